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
// angle's fraction of a turn exactly; its top 32 bits go through sincospif.  The error
// left is that of the fraction (2^-54 of a turn per position: 2^-32 at 4,194,304).
#include "ls_device.cuh"
#include "ls_internal.h"

namespace {

constexpr int kD = 128;
constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;  // half-warps; each works on one row at a time
constexpr int kMaxTok = 16;             // tokens of a block
constexpr int kMaxHalf = kD / 2;
constexpr float kOverflow = 3.0e38f;

// The angle table of a block's tokens: tab[tok][pair] = (cos, sin).
__device__ __forceinline__ void fill_angles(const LsNormRopeArgs& a, int64_t t0, int tb,
                                            float2 (*tab)[kMaxHalf]) {
  for (int i = threadIdx.x; i < tb * a.half; i += kThreads) {
    const int tok = i / a.half, j = i - tok * a.half;
    float2 cs = make_float2(1.f, 0.f);
    if (t0 + tok < a.T) {
      int ax = a.pair_axis ? __ldg(a.pair_axis + j) : 0;
      if ((uint32_t)ax >= (uint32_t)a.axes) {
        ls_report(a.err, LS_DEVERR_CHECK);
        ax = 0;
      }
      const double turns = __ldg(a.inv_freq + j) * 0.15915494309189533577;  // 1 / (2 pi)
      const unsigned long long f =
          __double2ull_rn((turns - floor(turns)) * 18446744073709551616.0);
      const long long p = __ldg(a.pos + (int64_t)ax * a.T + t0 + tok);
      const unsigned long long ph = (unsigned long long)p * f;
      sincospif((float)(int32_t)(ph >> 32) * 4.656612873077392578125e-10f, &cs.y, &cs.x);
    }
    tab[tok][j] = cs;
  }
}

// What a lane of a half-warp needs of the rotation of its eight values 8 l .. 8 l + 7.
struct Turn {
  float c[8], s[8];  // split halves: per value (s negated for the first of a pair)
  int partner;       // split: lane holding the other halves of the pairs
  bool active;       // the lane's values are rotated
};

__device__ __forceinline__ Turn load_turn(const LsNormRopeArgs& a, const float2* tab, int l,
                                          bool back) {
  Turn r;
  const int e0 = 8 * l;
  r.partner = l;
  r.active = e0 < 2 * a.half;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    r.c[i] = 1.f;
    r.s[i] = 0.f;
  }
  if (!r.active) return r;
  if (a.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 cs = tab[e0 / 2 + i];
      r.c[2 * i] = r.c[2 * i + 1] = cs.x;
      r.s[2 * i] = back ? cs.y : -cs.y;
      r.s[2 * i + 1] = back ? -cs.y : cs.y;
    }
  } else {
    const bool first = e0 < a.half;
    const int j0 = first ? e0 : e0 - a.half;
    r.partner = first ? l + a.half / 8 : l - a.half / 8;
    const bool neg = first != back;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 cs = tab[j0 + i];
      r.c[i] = cs.x;
      r.s[i] = neg ? -cs.y : cs.y;
    }
  }
  return r;
}

// y = u turned: every lane of the warp takes part.
__device__ __forceinline__ void turn8(const Turn& r, bool interleaved, float* u) {
  if (interleaved) {
    if (!r.active) return;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float x = u[i], y = u[i + 1];
      u[i] = fmaf(x, r.c[i], y * r.s[i]);
      u[i + 1] = fmaf(y, r.c[i + 1], x * r.s[i + 1]);
    }
  } else {
    const int src = (threadIdx.x & 16) | r.partner;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, u[i], src);
      if (r.active) u[i] = fmaf(u[i], r.c[i], o * r.s[i]);
    }
  }
}

__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// 1 / sqrt(mean x^2 + eps) of a row.  bf16 values reach 3e38, whose squares do not fit
// fp32: such a row is summed again scaled by 2^-80.
__device__ __forceinline__ float row_rstd(const float* x, float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
  ss = sum16(ss);
  float r = rsqrtf(fmaf(ss, 1.f / kD, eps));
  if (__any_sync(0xffffffffu, ss > kOverflow)) {
    float s2 = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = x[i] * 8.271806125530277e-25f;
      s2 = fmaf(y, y, s2);
    }
    s2 = sum16(s2);
    if (ss > kOverflow) r = rsqrtf(s2 * (1.f / kD)) * 8.271806125530277e-25f;
  }
  return r;
}

__device__ __forceinline__ void load_weights(const LsNormRopeArgs& a, int which, int l, float* w) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f;
  if (!a.norm || !a.w[which]) return;
  if (a.w_bf16) {
    unpack8(__ldg(static_cast<const uint4*>(a.w[which]) + l), w);
  } else {
    const float4* p = static_cast<const float4*>(a.w[which]) + 2 * l;
    const float4 x = __ldg(p), y = __ldg(p + 1);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    w[4] = y.x; w[5] = y.y; w[6] = y.z; w[7] = y.w;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] += a.w_offset;
}

// Forward.  A block takes `tb` tokens (a power of two up to 16); 16 / tb half-warps share
// a token and take its heads in turn, kRows rows' loads in flight each.
constexpr int kRows = 4;
template <bool kAppend>
__global__ void __launch_bounds__(kThreads)
norm_rope_fwd_kernel(const LsNormRopeArgs a, const LsRows x, const LsRows y, const LsPoolDst dst,
                     int tb) {
  __shared__ float2 tab[kMaxTok][kMaxHalf];
  const int l = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * tb;
  const int tok = grp % tb, sub = grp / tb, S = kGroups / tb;
  const int64_t t = t0 + tok;
  bool live = t < a.T;
  int64_t slot = 0;
  bool paged = true;
  if (kAppend && live) {
    const int32_t s = __ldg(dst.slots + t);
    live = s >= 0;  // a padding token: nothing of it is written
    paged = live && (s >> dst.ps_log2) < dst.num_pages;
    if (live && !paged) ls_report(a.err, LS_DEVERR_CHECK);
    slot = s;
  }
  float w[2][8];
  load_weights(a, 0, l, w[0]);
  load_weights(a, 1, l, w[1]);
  fill_angles(a, t0, tb, tab);
  __syncthreads();
  const Turn turn = load_turn(a, tab[tok], l, false);
#pragma unroll
  for (int which = 0; which < 3; ++which) {
    if (which == 2 && !x.p[2]) break;
    const int H = which == 0 ? a.hq : a.hkv;
    const uint4* src = static_cast<const uint4*>(x.p[which]) + t * (x.ts[which] >> 3) + l;
    const int64_t shs = x.hs[which] >> 3;
    uint4* out;
    int64_t ohs;
    bool write = live;
    if (kAppend && which > 0) {
      const int64_t ps = 1ll << dst.ps_log2;
      out = static_cast<uint4*>(which == 1 ? dst.k_pool : dst.v_pool) + l;
      if (paged) out += (((slot >> dst.ps_log2) * a.hkv << dst.ps_log2) + (slot & (ps - 1))) * 16;
      ohs = ps * 16;
      write = live && paged;
    } else {
      out = static_cast<uint4*>(const_cast<void*>(y.p[which])) + t * (y.ts[which] >> 3) + l;
      ohs = y.hs[which] >> 3;
    }
    for (int h0 = 0; h0 < H; h0 += S * kRows) {
      uint4 v[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int h = h0 + sub + i * S;
        v[i] = make_uint4(0, 0, 0, 0);
        if (write && h < H) v[i] = src[h * shs];
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int h = h0 + sub + i * S;
        if (h0 + i * S >= H) break;  // uniform over the block
        if (which < 2) {
          float u[8];
          unpack8(v[i], u);
          if (a.norm) {
            const float r = row_rstd(u, a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] = u[e] * r * w[which & 1][e];
          }
          turn8(turn, a.interleaved != 0, u);
          v[i] = pack8(u);
        }
        if (write && h < H) out[h * ohs] = v[i];
      }
    }
  }
}

// Backward.  The same blocks, walked by a persistent grid so that each lane keeps the
// weight gradients of its eight values in registers over all its rows; a block leaves
// one partial per weight, which norm_rope_dw sums in block order.
constexpr int kBwdRows = 2;

template <bool kBf16>
struct Grad8 {
  uint4 a, b;
};
template <bool kBf16>
__device__ __forceinline__ Grad8<kBf16> load_grad(const void* base, int64_t off, int l) {
  Grad8<kBf16> g;
  if (kBf16) {
    g.a = *(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off) + l);
    g.b = make_uint4(0, 0, 0, 0);
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + off) + 2 * l;
    g.a = p[0];
    g.b = p[1];
  }
  return g;
}
template <bool kBf16>
__device__ __forceinline__ void unpack_grad(const Grad8<kBf16>& g, float* x) {
  if (kBf16) {
    unpack8(g.a, x);
  } else {
    const uint32_t u[8] = {g.a.x, g.a.y, g.a.z, g.a.w, g.b.x, g.b.y, g.b.z, g.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
norm_rope_bwd_kernel(const LsNormRopeArgs a, const LsRows x, const LsRows dy, const LsRows dx,
                     float* part, int tb) {
  __shared__ float2 tab[kMaxTok][kMaxHalf];
  __shared__ float red[kGroups][kD];
  const int l = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int tok = grp % tb, sub = grp / tb, S = kGroups / tb;
  float w[2][8], dw[2][8];
  load_weights(a, 0, l, w[0]);
  load_weights(a, 1, l, w[1]);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;
  const int64_t nblk = (a.T + tb - 1) / tb;
  for (int64_t blk = blockIdx.x; blk < nblk; blk += gridDim.x) {
    const int64_t t0 = blk * tb, t = t0 + tok;
    const bool live = t < a.T;
    __syncthreads();  // the table's readers of the last block are done
    fill_angles(a, t0, tb, tab);
    __syncthreads();
    const Turn turn = load_turn(a, tab[tok], l, true);
#pragma unroll
    for (int which = 0; which < 3; ++which) {
      if (which == 2 && !dy.p[2]) break;
      const int H = which == 0 ? a.hq : a.hkv;
      const int64_t xo = t * x.ts[which], yo = t * dy.ts[which];
      const uint4* src = static_cast<const uint4*>(x.p[which]) + (xo >> 3) + l;
      uint4* out = static_cast<uint4*>(const_cast<void*>(dx.p[which])) + t * (dx.ts[which] >> 3) + l;
      for (int h0 = 0; h0 < H; h0 += S * kBwdRows) {
        uint4 v[kBwdRows];
        Grad8<kBf16> gr[kBwdRows];
#pragma unroll
        for (int i = 0; i < kBwdRows; ++i) {
          const int h = h0 + sub + i * S;
          v[i] = gr[i].a = gr[i].b = make_uint4(0, 0, 0, 0);
          if (live && h < H) {
            if (which < 2 && a.norm) v[i] = src[h * (x.hs[which] >> 3)];
            gr[i] = load_grad<kBf16>(dy.p[which], yo + h * dy.hs[which], l);
          }
        }
#pragma unroll
        for (int i = 0; i < kBwdRows; ++i) {
          const int h = h0 + sub + i * S;
          if (h0 + i * S >= H) break;  // uniform over the block
          float g[8];
          unpack_grad<kBf16>(gr[i], g);
          if (which < 2) {
            turn8(turn, a.interleaved != 0, g);
            if (a.norm) {
              float u[8];
              unpack8(v[i], u);
              const float r = row_rstd(u, a.eps);
              float dot = 0.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                u[e] *= r;
                dw[which & 1][e] = fmaf(g[e], u[e], dw[which & 1][e]);
                g[e] *= w[which & 1][e];
                dot = fmaf(g[e], u[e], dot);
              }
              dot = sum16(dot) * (1.f / kD);
#pragma unroll
              for (int e = 0; e < 8; ++e) g[e] = r * fmaf(-dot, u[e], g[e]);
            }
          }
          if (live && h < H) out[h * (dx.hs[which] >> 3)] = pack8(g);
        }
      }
    }
  }
  if (!part) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) red[grp][8 * l + i] = dw[which][i];
    __syncthreads();
    if (threadIdx.x < kD) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) s += red[i][threadIdx.x];
      part[((int64_t)blockIdx.x * 2 + which) * kD + threadIdx.x] = s;
    }
  }
}

// dw[c] (+)= sum over blocks of part[block][c], in block order within each of 32 strided
// chains, summed in 64 bits.  256 columns (queries, keys), 32 per block.
__global__ void __launch_bounds__(1024) norm_rope_dw(const float* __restrict__ part, int blocks,
                                                     float* dwq, float* dwk, int accumulate) {
  __shared__ double red[32][33];
  const int c = threadIdx.x & 31, chain = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  double s = 0.0;
  for (int b = chain; b < blocks; b += 32) s += part[(int64_t)b * 2 * kD + col];
  red[chain][c] = s;
  __syncthreads();
  if (chain) return;
  s = 0.0;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += red[i][c];
  float* dw = col < kD ? dwq : dwk;
  if (!dw) return;
  float* p = dw + (col & (kD - 1));
  *p = accumulate ? (float)(*p + s) : (float)s;
}

// Tokens of a block: the most (up to 16) that still give every SM four blocks.
int block_tokens(int64_t T, int sms) {
  int tb = kMaxTok;
  while (tb > 1 && T < (int64_t)tb * sms * 4) tb >>= 1;
  return tb;
}

}  // namespace

cudaError_t ls_launch_norm_rope_fwd(const LsNormRopeArgs& a, const LsRows& x, const LsRows& y,
                                    const LsPoolDst* dst, int sms, cudaStream_t st) {
  const int tb = block_tokens(a.T, sms);
  const int64_t blocks = (a.T + tb - 1) / tb;
  if (dst)
    norm_rope_fwd_kernel<true><<<(unsigned)blocks, kThreads, 0, st>>>(a, x, y, *dst, tb);
  else
    norm_rope_fwd_kernel<false><<<(unsigned)blocks, kThreads, 0, st>>>(a, x, y, LsPoolDst{}, tb);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ls_note_launch();
  return e;
}

int ls_norm_rope_bwd_ctas(int64_t T, int sms) {
  const int tb = block_tokens(T, sms);
  const int64_t blocks = (T + tb - 1) / tb, cap = (int64_t)sms * 4;
  return (int)(blocks < cap ? blocks : cap);
}

cudaError_t ls_launch_norm_rope_bwd(const LsNormRopeArgs& a, const LsRows& x, const LsRows& dy,
                                    int dy_bf16, const LsRows& dx, float* dwq, float* dwk,
                                    int accumulate, float* part, int sms, cudaStream_t st) {
  const int tb = block_tokens(a.T, sms), ctas = ls_norm_rope_bwd_ctas(a.T, sms);
  const bool dw = dwq || dwk;
  cudaError_t e = cudaSuccess;
  if (ctas > 0) {  // no tokens: zero weight gradients only
    if (dy_bf16)
      norm_rope_bwd_kernel<true><<<ctas, kThreads, 0, st>>>(a, x, dy, dx, dw ? part : nullptr, tb);
    else
      norm_rope_bwd_kernel<false><<<ctas, kThreads, 0, st>>>(a, x, dy, dx, dw ? part : nullptr, tb);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    ls_note_launch();
  }
  if (dw) {
    norm_rope_dw<<<2 * kD / 32, 1024, 0, st>>>(part, ctas, dwq, dwk, accumulate);
    e = cudaGetLastError();
    if (e == cudaSuccess) ls_note_launch();
  }
  return e;
}
