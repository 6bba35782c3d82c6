// decode_attn.cu -- decode attention of a group whose members share one captured prompt.
//
// Each member has n new tokens (one, or a few) whose keys and values are the last n of
// its response pages.  For token i of member m with len keys in its pages, query head h,
// KV head h / g:
//   s_j = scale <q, k_j> over the P prompt positions and the member's response keys
//         j <= len - n + i;   lse = log sum_j exp(s_j);   o = sum_j exp(s_j - lse) v_j
//
// Work.  A row tile is up to 128 rows (token, head of the group) that share a KV head:
// all members' tokens against the prompt's keys (each prompt K/V tile serves every
// member), one member's tokens against its own keys.  The prompt's tiles (128 keys, KV
// head by KV head) followed by the responses' tiles (member by member, KV head by KV
// head) form one sequence that is cut evenly over the grid, so a CTA holds a few
// segments, each a run of tiles of one row tile and one key source; a segment leaves a
// partial (o, lse) and decode_combine merges a row's partials by log-sum-exp.  With more
// rows than one tile (rts row tiles) the prompt part is cut over `cols` columns of rts
// CTAs: a column's CTAs walk the same prompt tiles at the same time, one row tile each, so
// a tile is read from HBM once and from L2 after that.  The response lengths stay on the
// device (a captured graph follows them): every CTA sums them when it starts.
//
// What bounds it.  A key and value row of 512 bytes meets at most 128 query rows, so the
// reads are the floor up to about 100 rows and the tensor core (1,024 clocks a tile, and
// 1,250 for the shared memory that feeds it) from there on.  Measured with 24 query and 4 KV
// heads, against the copy's 6,783 GB/s: 8 members over 2,097,152 tokens 625 us, the whole of
// it; 64 members with up to 8,192 tokens of their own over 262,139 tokens 243 us, 67%: there a
// tile takes 1,650 clocks, one after the other through a softmax warp (scores loaded, maximum,
// exchange, exponentials, weights stored and handed over); 2 members over 4,096 tokens (8 and 2
// heads) 11.5 us, the latency of two launches.
//
// CTA (one per SM, 12 warps):
//   warp 0      TMA producer of the segments' K tiles, page by page, into a ring of 3.
//   warp 1      issues S = Q K^T into one of two S buffers, as soon as the softmax has the
//               scores before the last ones in registers.
//   warp 2      issues O += P V, P read from one of two buffers in tensor memory.
//               (One thread for both kinds of MMA, and one for both kinds of load, were each
//               the bound with several row tiles: about 2,000 clocks a tile.)
//   warp 3      TMA producer of V; loads the segments' Q; clears the V rows behind a
//               sequence's end (stale page contents, even NaN, would survive a zero weight)
//               before such a tile is handed over.
//   warps 4-7   softmax of a tile's keys 0-63, warps 8-11 of its keys 64-127, one row a
//               thread.  The two threads of a row exchange their maxima through shared memory
//               and go by the larger; each rescales and writes out half of the row's O.
//               (As two sequences with an O each, P in the place of S, nothing is exchanged
//               but the next S waits for P V: 5 to 7% slower at 8 to 42 members of a few
//               tokens, 1% faster at 64 with long responses.  One warpgroup a tile, by turns,
//               was slower and spilled registers; the next tile's scores loaded before the
//               weights are stored were slower both ways.)
//               Warps whose rows are all padding only keep the barriers going.
// Tensor memory (512 columns): S_0 [0,128) S_1 [128,256) O [256,384) P_0 [384,448) P_1 [448,512).
#include <math.h>

#include "ls_decode.cuh"

namespace {

using namespace umma;
using namespace decode;

constexpr int kRing = 3;  // K tiles, and V tiles, in shared memory
constexpr int kThreads = 384;
constexpr int kSoftmaxThreads = 256;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kTileBytes;
constexpr uint32_t kOffV = kOffK + kRing * kTileBytes;
// A segment of up to 64 query rows takes half of the Q tile, by turns, so that the next
// segment's rows can be there before the last one is done.  Its MMAs still read 128 rows,
// the other half's or the ring's bytes among them: rows that nothing looks at.
constexpr int kHalfRows = kTile / 2;
constexpr uint32_t kOffBar = kOffV + kRing * kTileBytes;
constexpr uint32_t kOffMax = kOffBar + 512;       // [2][2][128] fp32: buffer, key half, row
constexpr uint32_t kSmemBytes = kOffMax + 2 * 2 * kTile * 4;
constexpr int kHalfKeys = kTile / 2;
constexpr uint32_t kColO = 2 * kTile, kColP = 3 * kTile;  // tensor memory behind the S buffers
constexpr int kSegTiles = 3;  // a segment's beginning and end take a CTA as long as so many tiles

enum {
  B_K_FULL = 0,
  B_K_EMPTY = B_K_FULL + kRing,
  B_V_FULL = B_K_EMPTY + kRing,
  B_V_EMPTY = B_V_FULL + kRing,  // P V of the tile is done
  B_AUX = B_V_EMPTY + kRing,     // a ragged V tile has landed, its tail not yet cleared
  B_Q_FULL = B_AUX + kRing,      // 2
  B_Q_EMPTY = B_Q_FULL + 2,      // 2
  B_S_FULL = B_Q_EMPTY + 2,      // 2: S buffers
  B_S_EMPTY = B_S_FULL + 2,      // 2: the scores are in registers
  B_P_FULL = B_S_EMPTY + 2,      // 2: P buffers
  B_PAIR = B_P_FULL + 2,         // 4: the two warps of 32 rows have shown their numbers
  B_O_DONE = B_PAIR + 4,
  B_DONE,                        // 2: the S and the P V issuer
  B_COUNT = B_DONE + 2
};
constexpr uint32_t kOffVars = kOffBar + B_COUNT * 8;
static_assert(B_COUNT * 8 + 32 <= 512, "barrier area");

__device__ __forceinline__ uint32_t bar_addr(uint32_t base, int i) { return base + kOffBar + 8 * i; }

// Units of the cut: the keys of one source under one KV head weigh their tiles and, in front
// of them, kSegTiles more.  (With tiles alone a CTA got up to 85 responses of one tile each
// at 64 members of a few tokens over 262,139: 317 us, with 1 more 247, with 2 180, with 3
// 176, with 5 190; at 8 members 142, 110, 97, 96, 97.  Each kind cut by itself, so that every
// CTA has its share of both, took 183 us for 169 there and 241 for 243 with long responses.)
__device__ __forceinline__ int32_t units_of(int32_t tiles) {
  return tiles > 0 ? tiles + kSegTiles : 0;
}

// The cut of the sequence.  A unit of the prompt occupies the rts CTAs of a column, a unit of
// a response one of them, so the sequence weighs rts tp + (responses' units).
struct Cut {
  int32_t tp, rts, cols;
  long long w;
  __device__ __forceinline__ Cut(const LsDecodeArgs& a, int32_t resp_units)
      : tp(units_of(a.nt) * a.hkv), rts(a.rts), cols(a.cols), w((long long)rts * tp + resp_units) {}
  __device__ __forceinline__ void prompt(int32_t col, int32_t* b, int32_t* e) const {
    *b = bound(col);
    *e = bound(col + 1);
  }
  __device__ __forceinline__ void resp(int32_t col, int32_t rt, int32_t* b, int32_t* e) const {
    const int32_t lo = rbound(col);
    const long long n = rbound(col + 1) - lo;
    *b = lo + (int32_t)(n * rt / rts);
    *e = lo + (int32_t)(n * (rt + 1) / rts);
  }

 private:
  __device__ __forceinline__ int32_t bound(int32_t col) const {
    const long long p = (w * col / cols + rts - 1) / rts;
    return p < tp ? (int32_t)p : tp;
  }
  __device__ __forceinline__ int32_t rbound(int32_t col) const {
    const long long r = w * col / cols - (long long)rts * tp;
    return r > 0 ? (int32_t)r : 0;
  }
};

// One segment: `count` tiles from key `key0` of one source; rows of one row tile.
struct Seg {
  bool resp;
  int32_t kvh, m;       // KV head; member (responses)
  int32_t item;         // KV head (prompt) or m * hkv + kvh
  int32_t key0, count;
  int32_t len;          // keys of the source
};

struct Walk {
  const LsDecodeArgs& a;
  int32_t p, p_end, r, r_end;
  int32_t m, off;       // member and unit within its KV heads' units
  __device__ __forceinline__ Walk(const LsDecodeArgs& a_, const volatile int32_t* start, int32_t p0,
                                  int32_t p1, int32_t r0, int32_t r1)
      : a(a_), p(p0), p_end(p1), r(r0), r_end(r1), m(start[0]), off(start[1]) {}
  __device__ __forceinline__ bool next(Seg* s) {
    while (p < p_end) {
      const int32_t nu = units_of(a.nt), h = p / nu, x = p - h * nu, step = min(p_end - p, nu - x);
      p += step;
      if (!tiles(s, x, step)) continue;
      s->resp = false;
      s->kvh = s->item = h;
      s->m = 0;
      s->len = (int32_t)a.P;
      return true;
    }
    while (r < r_end) {
      int32_t len = 0, nt = 0, nu = 0;
      for (; m < a.M; ++m, off = 0) {
        len = clamp_len(a, __ldg(a.lens + m));
        nt = tiles_of(len);
        nu = units_of(nt);
        if (off < nu * a.hkv) break;
      }
      if (m >= a.M) return false;  // only when lengths changed under the kernel
      const int32_t h = off / nu, x = off - h * nu, step = min(r_end - r, nu - x);
      r += step;
      off += step;
      if (!tiles(s, x, step)) continue;
      s->resp = true;
      s->kvh = h;
      s->m = m;
      s->item = m * a.hkv + h;
      s->len = len;
      return true;
    }
    return false;
  }

 private:
  // the tiles among units x .. x + step - 1 of a source; none: they are another CTA's
  __device__ __forceinline__ static bool tiles(Seg* s, int32_t x, int32_t step) {
    const int32_t first = max(x - kSegTiles, 0);
    s->key0 = first * kTile;
    s->count = x + step - kSegTiles - first;
    return s->count > 0;
  }
};

// Query rows of a segment: row r of row tile rt is row rt x 128 + r of all (token, head of
// the group) pairs against the prompt, row r of the member's own against a response.
__device__ __forceinline__ int32_t seg_rows(const LsDecodeArgs& a, const Seg& s, int32_t rt) {
  return s.resp ? a.n * a.g : min(a.M * a.n * a.g - rt * kTile, kTile);
}

__device__ __forceinline__ bool whole_q(const LsDecodeArgs& a, const Seg& s, int32_t rt) {
  return seg_rows(a, s, rt) > kHalfRows;
}
__device__ __forceinline__ uint32_t q_offset(bool whole, uint32_t seg) {
  return kOffQ + (whole ? 0u : (seg & 1) * kHalfRows * 128u);
}

// Rows of a partial: prompt partials first, then the responses'.  (item + CTA in walk
// order) numbers a CTA's segments uniquely: from one segment to the next of the whole
// sequence the item, the CTA or both grow.  Eight rows lie together, four values of each in
// turn: a warp of the main kernel, which has a row a lane, writes whole 128-byte lines, and a
// warp of the combine reads the rows of one KV head's group with whole sectors.  (Row by row,
// a warp's stores met 32 lines each and 128 rows took more than 4 us to write: 64 responses
// of up to 8,192 tokens took 123 us where this takes 103.  Transposed by shuffles instead,
// the group of 64 members below took 259 us for 246.)
__host__ __device__ __forceinline__ int32_t resp_rows_of(const LsDecodeArgs& a) {
  return (a.n * a.g + 7) & ~7;
}
__device__ __forceinline__ int64_t prompt_row0(const LsDecodeArgs& a, int32_t h, int32_t col,
                                               int32_t rt) {
  return (((int64_t)h + col) * a.rts + rt) * kTile;
}
__device__ __forceinline__ int64_t resp_row0(const LsDecodeArgs& a, int64_t prompt_rows,
                                             int32_t item, int32_t cta) {
  return prompt_rows + ((int64_t)item + cta) * resp_rows_of(a);
}
__host__ __device__ __forceinline__ int64_t prompt_rows_of(const LsDecodeArgs& a) {
  return a.nt > 0 ? ((int64_t)a.hkv + a.cols) * a.rts * kTile : 0;
}

template <bool kTree>
__global__ void __launch_bounds__(kThreads, 1)
decode_attn_kernel(const __grid_constant__ TmapSet tm, const __grid_constant__ LsDecodeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw;
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023) {  // the swizzled tiles' alignment, which the declaration asks for
    if (threadIdx.x == 0) ls_report(a.err, LS_DEVERR_CHECK);
    return;
  }
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kOffVars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffVars + 4);
  volatile int32_t* start = reinterpret_cast<volatile int32_t*>(smem + kOffVars + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t cta = blockIdx.x, col = cta / a.rts, rt = cta - col * a.rts;

  // the combine may be launched: its blocks wait for this grid before they read from it
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // ---- units of the responses before each member, summed by the whole CTA (scratch: the ring,
  // which no copy has touched yet)
  int32_t p0, p1, r0, r1;
  {
    int32_t* wsum = reinterpret_cast<int32_t*>(smem + kOffK);
    const int per = (a.M + kThreads - 1) / kThreads;
    int32_t mine = 0;
    for (int i = 0; i < per; ++i) {
      const int m = tid * per + i;
      if (m < a.M) {
        const int32_t len = __ldg(a.lens + m);
        const int32_t cl = clamp_len(a, len);
        if (cta == 0 && (kTree ? bad_member(a, m) : len > cl)) ls_report(a.err, LS_DEVERR_CHECK);
        mine += units_of(tiles_of(cl));
      }
    }
    int32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) wsum[warp] = sum;
    if (tid == 0) start[0] = start[1] = 0;
    __syncthreads();
    int32_t before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      const int32_t v = wsum[i];
      if (i < warp) before += v;
      total += v;
    }
    const Cut cut(a, total * a.hkv);
    cut.prompt(col, &p0, &p1);
    cut.resp(col, rt, &r0, &r1);
    // the member whose units hold r0
    int32_t pre = before + sum - mine;
    if (r0 < r1 && pre * a.hkv <= r0 && r0 < (pre + mine) * a.hkv) {
      for (int i = 0; i < per; ++i) {
        const int m = tid * per + i;
        const int32_t nu = units_of(tiles_of(clamp_len(a, __ldg(a.lens + m))));
        if (r0 < (pre + nu) * a.hkv) {
          start[0] = m;
          start[1] = r0 - pre * a.hkv;
          break;
        }
        pre += nu;
      }
    }
    if (p0 >= p1 && r0 >= r1) return;  // uniform: no tiles for this CTA
  }

  if (tid == 0) {
    for (int i = 0; i < B_Q_FULL; ++i) mbar_init(bar_addr(sbase, i), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_addr(sbase, B_Q_FULL + i), 1);
      mbar_init(bar_addr(sbase, B_Q_EMPTY + i), 1);
      mbar_init(bar_addr(sbase, B_S_FULL + i), 1);
      mbar_init(bar_addr(sbase, B_S_EMPTY + i), kSoftmaxThreads);
      mbar_init(bar_addr(sbase, B_P_FULL + i), kSoftmaxThreads);
    }
    for (int i = 0; i < 4; ++i) mbar_init(bar_addr(sbase, B_PAIR + i), kSoftmaxThreads / 4);
    mbar_init(bar_addr(sbase, B_O_DONE), 1);
    mbar_init(bar_addr(sbase, B_DONE), 1);
    mbar_init(bar_addr(sbase, B_DONE + 1), 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    tmem_relinquish();
  }
  fence_proxy_async_smem();  // the scratch above, before TMA writes the ring
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&](void) {
    ls_report(a.err, LS_DEVERR_TIMEOUT);
    *abort_flag = 1;
  };
  Walk walk(a, start, p0, p1, r0, r1);
  Seg s;

  if (warp == 0) {
    // ------------------------------------------------------------ K loads
    if (lane == 0) {
      tma_prefetch_desc(&tm.kp);
      tma_prefetch_desc(&tm.kr);
      RingPos<kRing> ring;
      uint32_t fills = 0;
      Loader ld;
      bool ok = true;
      while (ok && walk.next(&s)) {
        ld.open(a, s.resp, s.m, s.kvh, s.key0, s.len, &tm.kp, &tm.kr);
        for (int32_t j = 0; j < s.count; ++j) {
          ok = wait_bar(bar_addr(sbase, B_K_EMPTY + ring.stage), ring.phase ^ 1) && !*abort_flag;
          if (!ok) {
            fail();
            break;
          }
          ld.load(sbase + kOffK + ring.stage * kTileBytes, bar_addr(sbase, B_K_FULL + ring.stage),
                  j + 1 < s.count, a.err);
          ring.advance();
          ++fills;
        }
      }
      // Do not leave while loads into this CTA's shared memory may still be in flight.
      for (uint32_t i = fills > kRing ? fills - kRing : 0; i < fills; ++i)
        mbar_wait(bar_addr(sbase, B_K_FULL + i % kRing), (i / kRing) & 1);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ Q, V loads, V tails
    // Q goes into the operand layout (128-byte swizzle: chunk c of row r lies at chunk
    // c ^ (r & 7)), row by row, so that a row tile may begin inside a token.  Rows behind
    // the segment's keep what was there: a row of S, P and O depends on its own row of Q
    // only, and theirs are not written out.
    if (lane == 0) {
      tma_prefetch_desc(&tm.vp);
      tma_prefetch_desc(&tm.vr);
    }
    RingPos<kRing> ring;
    uint32_t fills = 0, aux_phase = 0, seg = 0;
    Loader ld;
    auto start_q = [&](uint32_t n_seg) {
      const int rows = seg_rows(a, s, rt);
      const uint32_t buf = sbase + q_offset(whole_q(a, s, rt), n_seg);
      const int32_t row0 = s.resp ? s.m * a.n * a.g : rt * kTile;
      int32_t token = (row0 + (lane >> 4)) / a.g, head = (row0 + (lane >> 4)) - token * a.g;
      const int c = lane & 15;
      for (int r = lane >> 4; r < rows; r += 2) {
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) +
                                   ((int64_t)token * a.hq + s.kvh * a.g + head) * kD + c * 8;
        cp_async16(buf + (c >> 3) * kHalfBytes + r * 128 + (((c & 7) ^ (r & 7)) << 4), src);
        for (head += 2; head >= a.g; head -= a.g) ++token;
      }
    };
    auto finish_q = [&](uint32_t n_seg) {
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_addr(sbase, B_Q_FULL + (n_seg & 1)));
    };
    bool ok = true, have = walk.next(&s);
    if (have) start_q(0);
    for (; ok && have; ++seg) {
      if (lane == 0) ld.open(a, s.resp, s.m, s.kvh, s.key0, s.len, &tm.vp, &tm.vr);
      uint32_t st = 0;
      for (int32_t j = 0; j < s.count; ++j) {
        st = ring.stage;
        ok = wait_bar(bar_addr(sbase, B_V_EMPTY + st), ring.phase ^ 1) && !*abort_flag;
        if (!ok) break;
        if (lane == 0) {
          const bool ragged = s.len - (s.key0 + j * kTile) < kTile;
          ld.load(sbase + kOffV + st * kTileBytes, bar_addr(sbase, (ragged ? B_AUX : B_V_FULL) + st),
                  j + 1 < s.count, a.err);
        }
        if (fills == 0) finish_q(0);
        ring.advance();
        ++fills;
      }
      if (!ok) break;
      const int32_t left = s.len - (s.key0 + (s.count - 1) * kTile);
      const bool whole = whole_q(a, s, rt);
      have = walk.next(&s);
      if (have) {
        // the next segment's Q: its half of the Q tile was the segment before's, and a whole
        // tile also waits for this one's last S
        if (seg > 0) ok = wait_bar(bar_addr(sbase, B_Q_EMPTY + ((seg - 1) & 1)), ((seg - 1) >> 1) & 1);
        if (ok && (whole || whole_q(a, s, rt)))
          ok = wait_bar(bar_addr(sbase, B_Q_EMPTY + (seg & 1)), (seg >> 1) & 1);
        if (!ok) break;
        start_q(seg + 1);
      }
      if (left < kTile) {  // the segment's last tile passes its source's end
        ok = wait_bar(bar_addr(sbase, B_AUX + st), (aux_phase >> st) & 1);
        if (!ok) break;
        aux_phase ^= 1u << st;
        uint8_t* vb = smem + kOffV + st * kTileBytes;
        for (int i = left * 8 + lane; i < kTile * 8; i += 32) {
          *reinterpret_cast<uint4*>(vb + i * 16) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(vb + kHalfBytes + i * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_addr(sbase, B_V_FULL + st));
      }
      if (have) finish_q(seg + 1);  // its rows came meanwhile
    }
    if (!ok) fail();
    cp_async_wait_all();
    for (uint32_t i = fills > kRing ? fills - kRing : 0; i < fills; ++i)
      mbar_wait(bar_addr(sbase, B_V_FULL + i % kRing), (i / kRing) & 1);
  } else if (warp == 1) {
    // ------------------------------------------------------------ S = Q K^T
    if (lane == 0) {
      const uint32_t idS = idesc_bf16_f32(kTile, kTile, false);
      const uint32_t dk = sdesc_lo(sbase + kOffK, 16);
      RingPos<kRing> ring;
      uint32_t n = 0, seg = 0;  // tiles, segments
      bool ok = true;
      for (; ok && walk.next(&s); ++seg) {
        ok = wait_bar(bar_addr(sbase, B_Q_FULL + (seg & 1)), (seg >> 1) & 1);
        const uint32_t dq = sdesc_lo(sbase + q_offset(whole_q(a, s, rt), seg), 16);
        for (int32_t j = 0; ok && j < s.count; ++j, ++n) {
          ok = wait_bar(bar_addr(sbase, B_K_FULL + ring.stage), ring.phase);
          if (ok && n >= 2) ok = wait_bar(bar_addr(sbase, B_S_EMPTY + (n & 1)), ((n - 2) >> 1) & 1);
          if (!ok || *abort_flag) break;
          tc_fence_after();
          const uint32_t b0 = dk + ((ring.stage * kTileBytes) >> 4), d_s = tmem + (n & 1) * kTile;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t off = ((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4;
            mma_ss_lo(d_s, dq + off, b0 + off, idS, kk > 0);
          }
          mma_commit(bar_addr(sbase, B_S_FULL + (n & 1)));
          mma_commit(bar_addr(sbase, B_K_EMPTY + ring.stage));
          if (j + 1 == s.count) mma_commit(bar_addr(sbase, B_Q_EMPTY + (seg & 1)));
          ring.advance();
        }
      }
      if (!ok) fail();
      // every MMA this thread issued has finished before tensor memory is released
      mma_commit(bar_addr(sbase, B_DONE));
      mbar_wait(bar_addr(sbase, B_DONE), 0);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ O += P V
    if (lane == 0) {
      const uint32_t idPV = idesc_bf16_f32(kTile, kD, true);
      const uint32_t dv = sdesc_lo(sbase + kOffV, kHalfBytes);
      RingPos<kRing> ring;
      uint32_t n = 0;
      bool ok = true;
      while (ok && walk.next(&s)) {
        for (int32_t j = 0; ok && j < s.count; ++j, ++n) {
          const uint32_t buf = n & 1, p_col = tmem + kColP + buf * kHalfKeys;
          const uint32_t b0 = dv + ((ring.stage * kTileBytes) >> 4);
          ok = wait_bar(bar_addr(sbase, B_V_FULL + ring.stage), ring.phase) &&
               wait_bar(bar_addr(sbase, B_P_FULL + buf), (n >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ts_lo(tmem + kColO, p_col + k * 8, b0 + ((k * 2048) >> 4), idPV, (j > 0 || k > 0) ? 1u : 0u);
          if (*abort_flag) break;
          if (j + 1 == s.count) mma_commit(bar_addr(sbase, B_O_DONE));
          mma_commit(bar_addr(sbase, B_V_EMPTY + ring.stage));
          ring.advance();
        }
      }
      if (!ok) fail();
      mma_commit(bar_addr(sbase, B_DONE + 1));
      mbar_wait(bar_addr(sbase, B_DONE + 1), 0);
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    const int t = (warp - 4) >> 2;  // half of a tile's keys
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t o_col = tmem + lane_off + kColO + t * kHalfKeys;  // this thread's half of O
    const float c = a.scale_log2;
    const int64_t prompt_rows = prompt_rows_of(a);
    volatile float* left = reinterpret_cast<volatile float*>(smem + kOffMax);
    uint32_t n = 0, oc = 0, pair = 0;
    RingPos<kRing> pv;  // of tile n - 2
    // the two threads of a row show each other a number, through slot `slot`
    auto exchange = [&](uint32_t slot, float x, float* other) {
      left[(slot * 2 + t) * kTile + row] = x;
      mbar_arrive(bar_addr(sbase, B_PAIR + quad));
      const bool met = wait_bar(bar_addr(sbase, B_PAIR + quad), pair & 1);
      ++pair;
      *other = left[(slot * 2 + 1 - t) * kTile + row];
      return met;
    };
    bool ok = true;
    while (ok && walk.next(&s)) {
      const int32_t rows = seg_rows(a, s, rt);
      const bool idle = quad * 32 >= rows;  // the whole warp is padding
      // keys of the half tile from its first one on that this row sees
      int32_t lim = (s.resp && !kTree ? min(s.len, s.len - a.n + 1 + row / a.g) : s.len) - s.key0 -
                    t * kHalfKeys;
      // of a tree's response: lim counts the member's context, which every row sees
      int32_t pad = 0;
      const uint32_t* bits = nullptr;
      if (kTree && s.resp) {
        pad = a.n - drafted_of(a, s.m);
        lim -= a.n - pad;
        bits = a.visible + ((int64_t)s.m * a.n + min(row / a.g, a.n - 1)) * a.words;
      }
      float m = -INFINITY, l = 0.f, lcomp = 0.f;
      for (int32_t j = 0; j < s.count; ++j, ++n, lim -= kTile) {
        const uint32_t buf = n & 1, s_col = tmem + lane_off + buf * kTile + t * kHalfKeys;
        ok = wait_bar(bar_addr(sbase, B_S_FULL + buf), (n >> 1) & 1);
        if (!ok) break;
        const uint32_t free_bar = bar_addr(sbase, B_V_EMPTY + pv.stage), free_phase = pv.phase;
        if (n >= 2) pv.advance();
        if (idle) {  // P keeps what was there: rows of D depend on their own rows of A only
          mbar_arrive(bar_addr(sbase, B_S_EMPTY + buf));
          // or the arrivals of two tiles would count for one
          ok = n < 2 || wait_bar(free_bar, free_phase);
          if (!ok) break;
          mbar_arrive(bar_addr(sbase, B_P_FULL + buf));
          continue;
        }
        tc_fence_after();
        uint32_t sr[64];
        tmem_ld32(s_col, sr);
        tmem_ld32(s_col + 32, sr + 32);
        tmem_wait_ld();
        reg_fence32(sr);
        reg_fence32(sr + 32);
        tc_fence_before();
        mbar_arrive(bar_addr(sbase, B_S_EMPTY + buf));
        if (kTree && s.resp) {
          if (lim < kHalfKeys) {  // drafted keys among these
            const uint64_t see = tree_window(a, bits, pad - lim, pad);
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (!((uint32_t)(see >> (e & 32)) & (1u << (e & 31)))) sr[e] = __float_as_uint(-INFINITY);
          }
        } else if (lim < kHalfKeys) {  // the source's ragged end, the causal end
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (e >= lim) sr[e] = __float_as_uint(-INFINITY);
        }
        float mx4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mx4[k] = fmaxf(__uint_as_float(sr[k]), __uint_as_float(sr[k + 4]));
#pragma unroll
        for (int e = 8; e < 64; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx4[k] = fmax3(mx4[k], __uint_as_float(sr[e + k]), __uint_as_float(sr[e + 4 + k]));
        float mt = fmaxf(fmax3(mx4[0], mx4[1], mx4[2]), mx4[3]) * c;
        float other;
        ok = exchange(buf, mt, &other);
        if (!ok) break;
        mt = fmaxf(mt, other);
        // the P buffer's last weights have been multiplied, most likely: asked here, needed
        // when the next ones are there
        const bool freed = n < 2 || mbar_try_wait(free_bar, free_phase);
        bool rescale = false;
        float alpha = 1.f;
        if (j == 0) {
          m = mt;
        } else if (mt > m + kRescaleLog2) {
          alpha = fast_exp2(m - mt);
          m = mt;
          l *= alpha;
          lcomp *= alpha;
          rescale = true;
        }
        const float msub = (m == -INFINITY) ? 0.f : m;
        if (__any_sync(0xffffffffu, rescale)) {
          // P V of the tile before may still be adding to O
          ok = mbar_wait(bar_addr(sbase, B_V_EMPTY + (n - 1) % kRing), ((n - 1) / kRing) & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < kHalfKeys; c0 += 32) {
            uint32_t ov[32];
            tmem_ld32(o_col + c0, ov);
            tmem_wait_ld();
            reg_fence32(ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(o_col + c0, ov);
          }
        }
        const float2 c2 = make_float2(c, c), nm2 = make_float2(-msub, -msub);
        float2 ls4[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                         make_float2(0.f, 0.f)};
        uint32_t pk[32];
#pragma unroll
        for (int jj = 0; jj < 32; ++jj) {
          float2 x = __ffma2_rn(
              make_float2(__uint_as_float(sr[2 * jj]), __uint_as_float(sr[2 * jj + 1])), c2, nm2);
          x.x = fast_exp2(x.x);
          x.y = fast_exp2(x.y);
          ls4[jj & 3] = __fadd2_rn(ls4[jj & 3], x);
          // weights in [0, 2^8] enter the product as bf16, as in the replay forward: their
          // roundings are independent, so o's error is that of one bf16 rounding
          pk[jj] = pack_bf16(x.x, x.y);
        }
        if (!__all_sync(0xffffffffu, freed)) {
          ok = mbar_wait(free_bar, free_phase);
          if (!ok) break;
        }
        tc_fence_after();
        tmem_st32(tmem + lane_off + kColP + buf * kHalfKeys + t * (kHalfKeys / 2), pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar_addr(sbase, B_P_FULL + buf));
        const float2 lsa = __fadd2_rn(__fadd2_rn(ls4[0], ls4[1]), __fadd2_rn(ls4[2], ls4[3]));
        const float ls = lsa.x + lsa.y;
        const float tsum = l + ls;
        lcomp += (l - tsum) + ls;
        l = tsum;
      }
      ok = ok && mbar_wait(bar_addr(sbase, B_O_DONE), oc & 1);
      if (!ok) break;
      ++oc;
      if (!idle) {
        float lt = l + lcomp, lo;
        ok = exchange((n - 1) & 1, lt, &lo);  // that slot's maxima have long been read
        if (!ok) break;
        lt = t ? lo + lt : lt + lo;
        tc_fence_after();
        const float inv = lt == 0.f ? 0.f : 1.f / lt;  // a row that sees no key here
        const int64_t prow =
            (s.resp ? resp_row0(a, prompt_rows, s.item, cta) : prompt_row0(a, s.item, col, rt)) + row;
        float* po = part_at(a, prow) + t * kHalfKeys * 8;
#pragma unroll 1
        for (int c0 = 0; c0 < kHalfKeys; c0 += 32) {
          uint32_t ov[32];
          tmem_ld32(o_col + c0, ov);
          tmem_wait_ld();
          reg_fence32(ov);
          if (row < rows) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(po + (c0 + i) * 8) =
                  make_float4(__uint_as_float(ov[i]) * inv, __uint_as_float(ov[i + 1]) * inv,
                              __uint_as_float(ov[i + 2]) * inv, __uint_as_float(ov[i + 3]) * inv);
          }
        }
        if (row < rows && t == 0) a.part_lse[prow] = lt == 0.f ? -INFINITY : m + log2f(lt);
        tc_fence_before();
      }
      if (*abort_flag) break;
    }
    if (!ok) fail();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Merge a row's partials: lse = log2 sum 2^lse_k, o = sum 2^(lse_k - lse) o_k, in a fixed
// order.  A block takes up to eight heads of one token and KV head, whose partials lie in the
// same columns and CTAs, and 32 of their 128 values; a lane has the values of one head.  Its
// eight warps take the partials by turns (at 2,097,152 tokens and 4 KV heads there are 76
// columns' worth), four at a time with a running maximum, so that nothing waits for the
// maximum of all; then the warps' sums are merged.  Which columns and CTAs meet the keys, a
// thread looks at one of each, needs only the lengths, so the launch overlaps the main
// kernel's end and waits for it then.
constexpr int kCombineThreads = 256;
constexpr int kCombineWarps = kCombineThreads / 32;

template <bool kTree>
__global__ void __launch_bounds__(kCombineThreads)
decode_combine(const __grid_constant__ LsDecodeArgs a) {
  __shared__ __align__(16) float acc[kCombineWarps][2][32][4];
  __shared__ int32_t sums[2][kCombineWarps];
  __shared__ float red[2][kCombineWarps][8];     // maximum, sum; by warp and head
  __shared__ uint16_t from[2][kCombineThreads];  // columns, CTAs with partials of the rows
  __shared__ int32_t counts[2][kCombineWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t octets = (a.g + 7) >> 3, group = (blockIdx.x >> 2) / octets;
  const int32_t head0 = 8 * ((blockIdx.x >> 2) - group * octets), col0 = 32 * (blockIdx.x & 3);
  const int32_t token = group / a.hkv, kvh = group - token * a.hkv, m = token / a.n;
  const int32_t len = __ldg(a.lens + m);
  if (len < 0 || (kTree && token - m * a.n < a.n - drafted_of(a, m))) {
    // A member out of use, or a token that is padding: its rows stay as they were.  Its blocks wait all the same: the
    // stream goes on when this grid ends, and with every member out of use nothing else
    // would hold it back until the main kernel has ended.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int32_t nt = tiles_of(clamp_len(a, len));
  int32_t tot = 0, pre = 0;
  for (int i = tid; i < a.M; i += kCombineThreads) {
    const int32_t x = units_of(tiles_of(clamp_len(a, __ldg(a.lens + i))));
    tot += x;
    if (i < m) pre += x;
  }
  tot = __reduce_add_sync(0xffffffffu, tot);
  pre = __reduce_add_sync(0xffffffffu, pre);
  if (lane == 0) {
    sums[0][warp] = tot;
    sums[1][warp] = pre;
  }
  __syncthreads();
  tot = pre = 0;
#pragma unroll
  for (int i = 0; i < kCombineWarps; ++i) {
    tot += sums[0][i];
    pre += sums[1][i];
  }
  const Cut cut(a, tot * a.hkv);
  bool hit[2] = {false, false};
  {
    const int32_t pb = kvh * units_of(a.nt) + kSegTiles, rb = pre * a.hkv + kvh * units_of(nt) + kSegTiles;
    int32_t b, e;
    if (tid < a.cols) {
      cut.prompt(tid, &b, &e);
      hit[0] = max(b, pb) < min(e, pb + a.nt);
    }
    if (tid < a.cols * a.rts) {
      cut.resp(tid / a.rts, tid % a.rts, &b, &e);
      hit[1] = max(b, rb) < min(e, rb + nt);
    }
  }
  uint32_t in_warp[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    in_warp[i] = __ballot_sync(0xffffffffu, hit[i]);
    if (lane == 0) counts[i][warp] = __popc(in_warp[i]);
  }
  __syncthreads();
  int32_t all[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    int32_t at = __popc(in_warp[i] & ((1u << lane) - 1));
#pragma unroll
    for (int v = 0; v < kCombineWarps; ++v) {
      if (v < warp) at += counts[i][v];
      all[i] += counts[i][v];
    }
    if (hit[i]) from[i][at] = (uint16_t)tid;
  }
  __syncthreads();
  const int32_t np = all[0], count = np + all[1];
  // a lane's head (behind the last one: that one again): row of all rows (token, head of the
  // group) against the prompt, row of the member's own
  const int32_t grow = token * a.g + min(head0 + (lane & 7), a.g - 1), mrow = grow - m * a.n * a.g;
  const int64_t prompt0 = prompt_row0(a, kvh, 0, grow / kTile) + grow % kTile;
  const int64_t resp0 = resp_row0(a, prompt_rows_of(a), m * a.hkv + kvh, 0) + mrow;
  const int32_t resp_rows = resp_rows_of(a);
  auto part_row = [&](int k) {
    if (k < np) return prompt0 + (int64_t)from[0][k] * a.rts * kTile;
    return resp0 + (int64_t)from[1][k - np] * resp_rows;
  };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kBatch = 4;
  float mx = -INFINITY, sum = 0.f;
  float4 s[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int k0 = warp; k0 < count; k0 += kBatch * kCombineWarps) {
    float l[kBatch], top = mx;
    float4 v[kBatch][2];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int k = k0 + i * kCombineWarps;
      l[i] = -INFINITY;
      if (k < count) {
        const int64_t row = part_row(k);
        const float* p = part_at(a, row) + (col0 / 4 + (lane >> 3)) * 32;
        l[i] = __ldcg(a.part_lse + row);
        v[i][0] = __ldcg(reinterpret_cast<const float4*>(p));
        v[i][1] = __ldcg(reinterpret_cast<const float4*>(p + 128));
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) top = fmaxf(top, l[i]);
    const float sub = top == -INFINITY ? 0.f : top, keep = exp2f(mx - sub);
    mx = top;
    sum *= keep;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      s[h] = make_float4(s[h].x * keep, s[h].y * keep, s[h].z * keep, s[h].w * keep);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float w = exp2f(l[i] - sub);
      sum += w;
      if (l[i] == -INFINITY) continue;  // a part that saw no key adds nothing
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s[h].x = fmaf(w, v[i][h].x, s[h].x);
        s[h].y = fmaf(w, v[i][h].y, s[h].y);
        s[h].z = fmaf(w, v[i][h].z, s[h].z);
        s[h].w = fmaf(w, v[i][h].w, s[h].w);
      }
    }
  }
  *reinterpret_cast<float4*>(acc[warp][0][lane]) = s[0];
  *reinterpret_cast<float4*>(acc[warp][1][lane]) = s[1];
  if (lane < 8) {
    red[0][warp][lane] = mx;
    red[1][warp][lane] = sum;
  }
  __syncthreads();
  // a thread a value: four values of eight heads a warp
  const int h = lane & 7, e = lane >> 3;
  if (head0 + h >= a.g) return;
  mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < kCombineWarps; ++i) mx = fmaxf(mx, red[0][i][h]);
  const float sub = mx == -INFINITY ? 0.f : mx;
  sum = 0.f;
  float o = 0.f;
#pragma unroll
  for (int i = 0; i < kCombineWarps; ++i) {
    const float w = exp2f(red[0][i][h] - sub);
    sum = fmaf(w, red[1][i][h], sum);
    o = fmaf(w, acc[i][warp >> 2][(warp & 3) * 8 + h][e], o);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key at all: o = 0, lse = -inf
  const int64_t row = (int64_t)token * a.hq + kvh * a.g + head0 + h;
  static_cast<__nv_bfloat16*>(a.o)[row * kD + col0 + warp * 4 + e] = __float2bfloat16_rn(o * inv);
  if (warp == 0 && e == 0 && col0 == 0) a.lse[row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

}  // namespace

int ls_decode_row_tile() { return kTile; }
int ls_decode_seg_tiles() { return kSegTiles; }
int64_t ls_decode_prompt_rows(const LsDecodeArgs& a) { return prompt_rows_of(a); }
int64_t ls_decode_resp_rows(const LsDecodeArgs& a) {
  return ((int64_t)a.M * a.hkv + (int64_t)a.cols * a.rts) * resp_rows_of(a);
}

namespace {

template <bool kTree>
cudaError_t launch(const LsDecodeArgs& a, cudaStream_t st) {
  TmapSet tm;
  if (!make_tmaps(a, &tm)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(decode_attn_kernel<kTree>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemBytes);
  if (e != cudaSuccess) return e;
  decode_attn_kernel<kTree><<<a.cols * a.rts, kThreads, kSmemBytes, st>>>(tm, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  ls_note_launch();
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.M * a.n * a.hkv * ((a.g + 7) / 8) * 4));
  cfg.blockDim = dim3(kCombineThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, decode_combine<kTree>, a);
  if (e == cudaSuccess) ls_note_launch();
  return e;
}

}  // namespace

cudaError_t ls_launch_decode_attn(const LsDecodeArgs& a, cudaStream_t st) {
  return a.visible ? launch<true>(a, st) : launch<false>(a, st);
}
