// tree_attn.cu -- decode attention of drafted trees with more rows than one tile a KV head.
//
// The last drafted[m] of member m's n rows are its draft.  For such a row, query head h, KV
// head h / g:
//   s_j = scale <q, k_j> over the P prompt positions, the member's context (its keys before the
//         draft) and the drafted keys whose bits are set for the row;
//   lse = log sum_j exp(s_j);   o = sum_j exp(s_j - lse) v_j
//
// Work.  The rows (drafted token, head of the group) of all members that share a KV head, padding
// left out, lie one behind the other and make pairs of row tiles of 128; a CTA takes a pair
// through a run of key tiles of 128, so that a K/V tile in shared memory serves 256 rows, and
// one tile's softmax runs beside the other's products.  A prompt item is a pair and one of S
// equal strips of a KV head's prompt; items go round the first `cp` CTAs, pairs first, so the
// CTAs of a round walk the same strips at the same time and a key tile comes from HBM about once.
// The responses' key tiles (member by member, pair of its rows, KV head) are cut evenly over the
// other CTAs.  cp and S are what makes the longer of the two shortest; every CTA works them out
// from the lengths and counts on the device, so a captured graph follows them.  Every segment
// leaves a partial (o, lse); tree_combine merges a row's partials by log-sum-exp.
//
// What bounds it.  256 rows meet a key tile of 64 KB for 4.2 MFLOP of each product: the tensor
// core, 2,048 clocks a step of two row tiles and 128 keys.  A step takes about 3,150: from one row
// tile's S to the other's lie the softmax's wake, its load of S and the issuer's wake.  8 members'
// 16 tokens of 24 / 4 heads over 2,097,152: 2.0 to 2.1 ms, 1,560 to 1,640 TFLOP/s (2.2 to 2.3 when
// repeated for seconds, at the power limit); 64 members of up
// to 24 over 32,749, with responses of up to 8,192: 410 us.  (S and P over one another, an S buffer a
// row tile: 2.31 ms.  Slots of 64 keys, two a row tile: 2.96 ms.)
//
// CTA (one per SM, 12 warps):
//   warp 0      TMA producer: K and V tiles, page by page, into a ring of five.
//   warps 1, 2  issue S_t = Q_t K^T and O_t += P_t V of tile A and tile B, one thread each.
//   warp 3      clears V rows behind a sequence's end (stale page contents, even NaN, would
//               survive a zero weight).
//   warps 4-7   softmax of tile A, warps 8-11 of tile B: a thread a row; they gather the next
//               segment's Q rows by token and head while the last P V runs.
// Tensor memory (512 columns): S [0,128) P_A [128,192) P_B [192,256) O_A [256,384) O_B [384,512).
// The tiles take the S buffer in turn: it is free as soon as the softmax has S in its registers, so
// a tile's next S is ready while its softmax still works on the last, and P V follows behind.
#include "ls_decode.cuh"

namespace {

using namespace umma;
using namespace decode;

constexpr int kPair = 2 * kTile;
constexpr int kMaxMembers = 1024;
constexpr int kStages = 5;
// K and V tiles: groups of eight rows, in each both halves (64 values a row)
constexpr uint32_t kGroup = 2048, kGroupHalf = 1024;
constexpr int kThreads = 384;
constexpr int kWarps = kThreads / 32;
// 384 x 168 registers at launch; 128 x 96 + 256 x 200 = 63,488 of the 64,512
constexpr int kRegsLaunch = 168, kRegsControl = 96, kRegsSoftmax = 200;
static_assert(128 * kRegsControl + 256 * kRegsSoftmax <= kThreads * kRegsLaunch, "register split");
constexpr uint32_t kOffQ = 0;  // Q_A, Q_B
constexpr uint32_t kOffRing = 2 * kTileBytes;
constexpr uint32_t kOffBar = kOffRing + kStages * kTileBytes;
constexpr uint32_t kColP = kTile, kColO = 2 * kTile;  // tensor memory behind the S buffer
constexpr int kSegTiles = 3;  // a segment's beginning and end take a CTA as long as so many tiles
constexpr int kRounds = 3;    // of prompt items that are tried

enum {
  B_KV_FULL = 0,
  B_KV_EMPTY = B_KV_FULL + kStages,
  B_AUX = B_KV_EMPTY + kStages,      // a ragged V tile has landed, its tail not yet cleared
  B_Q_FULL = B_AUX + kStages,  // 2
  B_S_FULL = B_Q_FULL + 2,   // 2
  B_S_TAKEN = B_S_FULL + 2,  // 2: S is in the softmax's registers (segments of two row tiles)
  B_S_ALONE = B_S_TAKEN + 2, // the same where tile A is alone
  B_P_FULL,                  // 2
  B_O_DONE = B_P_FULL + 2,   // 2
  B_DONE = B_O_DONE + 2,     // 2
  B_PV_DONE = B_DONE + 2,    // 2
  B_COUNT = B_PV_DONE + 2
};

// How the work is cut, from the members' lengths and drafts.
struct Plan {
  int32_t tokens;   // drafted ones of all members
  int32_t np;       // pairs of row tiles against the prompt
  int32_t strips, strip;  // of the prompt, and a strip's tiles
  int32_t cp;       // CTAs of the prompt
  int32_t units, rcs;  // of the responses, and their CTAs: at least a unit each
  int32_t m0, off0;  // response CTAs: the member its first unit lies with, and how far in
};
// What the combine reads of it (workspace): also the tokens before each member and, for every
// pair of a member's rows and KV head, the first and the last response CTA that has some of its
// tiles.
struct Out {
  Plan plan;
  int32_t tok[kMaxMembers];
};
__device__ __forceinline__ int32_t* cta_range(const LsDecodeArgs& a, int32_t m, int32_t pair, int32_t h);
struct Vars {
  uint32_t tmem;
  int32_t abort;
  Plan plan;
  unsigned long long best;
};
constexpr uint32_t kOffVars = kOffBar + B_COUNT * 8;
constexpr uint32_t kOffTok = kOffBar + 512;  // tokens before each member
constexpr uint32_t kSmemBytes = kOffTok + (kMaxMembers + 2) * 2;
static_assert(B_COUNT * 8 + sizeof(Vars) <= 512 && kOffVars % 8 == 0, "barrier area");
static_assert(kSmemBytes <= 232448, "shared memory");

__device__ __forceinline__ uint32_t bar_addr(uint32_t base, int i) { return base + kOffBar + 8 * i; }

__device__ __forceinline__ int32_t pairs_of(const LsDecodeArgs& a, int32_t tokens) {
  return (tokens * a.g + kPair - 1) / kPair;
}
// Units of a member: for every pair of its rows and KV head its key tiles and, in front of them,
// kSegTiles more.
__device__ __forceinline__ int32_t item_units(const LsDecodeArgs& a, int32_t m) {
  return tiles_of(clamp_len(a, __ldg(a.lens + m))) + kSegTiles;
}
__device__ __forceinline__ int32_t member_units(const LsDecodeArgs& a, int32_t m, int32_t c) {
  if (c == 0 || clamp_len(a, __ldg(a.lens + m)) == 0) return 0;
  return pairs_of(a, c) * a.hkv * item_units(a, m);
}
__host__ __device__ __forceinline__ int32_t max_pairs(const LsDecodeArgs& a) {
  return (a.n * a.g + kPair - 1) / kPair;
}
__host__ __device__ __forceinline__ int32_t resp_rows_of(const LsDecodeArgs& a) {
  const int32_t r = (a.n * a.g + 7) & ~7;
  return r < kPair ? r : kPair;
}
// Rows of partials: 256 a prompt item, then a row group's a response segment.  (Item + CTA
// numbers a CTA's response segments uniquely: from one to the next of the whole sequence the
// item, the CTA or both grow.)
__host__ __device__ __forceinline__ int64_t prompt_rows_of(const LsDecodeArgs& a) {
  if (a.nt == 0) return 0;
  const int64_t np = ((int64_t)a.M * a.n * a.g + kPair - 1) / kPair * a.hkv;
  const int64_t most = (int64_t)kRounds * a.cols;
  return (np > most ? np : most) * kPair;
}
__device__ __forceinline__ int32_t* cta_range(const LsDecodeArgs& a, int32_t m, int32_t pair, int32_t h) {
  return reinterpret_cast<int32_t*>(static_cast<Out*>(a.plan) + 1) + 2 * ((m * max_pairs(a) + pair) * a.hkv + h);
}
__device__ __forceinline__ int64_t resp_row0(const LsDecodeArgs& a, int32_t m, int32_t pair, int32_t h,
                                             int32_t rc) {
  const int32_t item = (m * max_pairs(a) + pair) * a.hkv + h;
  return prompt_rows_of(a) + ((int64_t)item + rc) * resp_rows_of(a);
}
__device__ __forceinline__ int32_t unit_bound(int32_t units, int32_t rc, int32_t n) {
  return (int32_t)((long long)units * rc / n);
}

// One segment: `count` key tiles from key0 on of one source, for `rows` rows of a pair.
struct Seg {
  bool resp;
  int32_t kvh, m;       // KV head; member (responses)
  int32_t row0, rows;   // the pair's first row (of all, or of the member's drafted ones)
  int32_t key0, count, len;
  int64_t part;         // first row of its partial
  __device__ __forceinline__ bool two() const { return rows > kTile; }
};

struct Walk {
  const LsDecodeArgs& a;
  const volatile Plan& p;
  const uint16_t* tok;
  int32_t at, end, m, off;
  bool resp;
  __device__ __forceinline__ Walk(const LsDecodeArgs& a_, const volatile Plan& p_, const uint16_t* tok_, int32_t cta)
      : a(a_), p(p_), tok(tok_), m(0), off(0), resp(cta >= p_.cp) {
    if (resp) {
      const bool some = cta - p.cp < p.rcs;
      at = some ? unit_bound(p.units, cta - p.cp, p.rcs) : 0;
      end = some ? unit_bound(p.units, cta - p.cp + 1, p.rcs) : 0;
      m = p.m0;
      off = p.off0;
    } else {
      at = cta;
      end = p.strips * p.np * a.hkv;
    }
  }
  __device__ __forceinline__ bool next(Seg* s, int32_t cta) {
    s->resp = resp;
    if (!resp) {
      if (at >= end) return false;
      const int32_t q = at / p.np, pair = at - q * p.np, h = q / p.strips, strip = q - h * p.strips;
      s->kvh = h;
      s->m = 0;
      s->row0 = pair * kPair;
      s->rows = min(p.tokens * a.g - s->row0, kPair);
      s->key0 = strip * p.strip * kTile;
      s->count = min(p.strip, a.nt - strip * p.strip);
      s->len = (int32_t)a.P;
      s->part = (int64_t)at * kPair;
      at += p.cp;
      return true;
    }
    while (at < end) {
      for (; m < a.M; ++m, off = 0)
        if (off < member_units(a, m, tok[m + 1] - tok[m])) break;
      if (m >= a.M) return false;  // only when lengths changed under the kernel
      const int32_t iu = item_units(a, m), item = off / iu, x = off - item * iu, step = min(end - at, iu - x);
      at += step;
      off += step;
      const int32_t first = max(x - kSegTiles, 0);  // its tiles among units x .. x + step - 1
      s->count = x + step - kSegTiles - first;
      if (s->count <= 0) continue;  // they are another CTA's
      const int32_t pair = item / a.hkv;
      s->kvh = item - pair * a.hkv;
      s->m = m;
      s->row0 = pair * kPair;
      s->rows = min((tok[m + 1] - tok[m]) * a.g - s->row0, kPair);
      s->key0 = first * kTile;
      s->len = clamp_len(a, __ldg(a.lens + m));
      s->part = resp_row0(a, m, pair, s->kvh, cta - p.cp);
      return true;
    }
    return false;
  }
};

// The loads of a segment's tiles, by a warp: a lane a page (from grouped maps, one copy each), which
// it looks up while the last tile's loads are under way.
struct Pages {
  const int32_t* table;
  int32_t len, key, box_rows, boxes, ps_log2, pages, head, pool_groups, page;

  // lane's page of the tile at first
  __device__ __forceinline__ void open(const LsDecodeArgs& a, const Seg& s, int lane) {
    table = s.resp ? a.blocks + (int64_t)s.m * a.max_blocks : a.page_table;
    ps_log2 = s.resp ? a.r_ps_log2 : a.ps_log2;
    pages = s.resp ? a.r_num_pages : a.num_pages;
    box_rows = min(1 << ps_log2, kTile);
    boxes = kTile / box_rows;
    pool_groups = ((pages * a.hkv) << ps_log2) >> 3;
    head = a.hkv;
    len = s.len;
    key = s.key0 + lane * box_rows;
    if (lane < boxes) look_up();
  }
  __device__ __forceinline__ void look_up() {
    if (key < len) page = __ldg(table + (key >> ps_log2));
  }
  __device__ __forceinline__ void issue(const void* map, int32_t kvh, uint32_t dst, uint32_t bar, int lane,
                                        uint32_t* err) const {
    if (lane == 0) mbar_expect_tx(bar, kTileBytes);
    __syncwarp();
    if (lane >= boxes) return;
    int32_t y = pool_groups;  // out of bounds: zero fill
    if (key < len) {
      if ((uint32_t)page < (uint32_t)pages)
        y = (((page * head + kvh) << ps_log2) + (key & ((1 << ps_log2) - 1))) >> 3;
      else
        ls_report(err, LS_DEVERR_CHECK);
    }
    tma_load_4d(dst + lane * box_rows * 256, map, 0, 0, 0, y, bar);
  }
  __device__ __forceinline__ void advance(bool more, int lane) {
    key += kTile;
    if (more && lane < boxes) look_up();
  }
};

// The plan, by all threads of a CTA (scratch: 2 x kWarps ints).
__device__ void make_plan(const LsDecodeArgs& a, Vars* v, uint16_t* tok, int32_t* scratch, int32_t cta) {
  Out* out = static_cast<Out*>(a.plan);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (a.M + kThreads - 1) / kThreads;
  int32_t tokens = 0, units = 0;
  for (int i = 0; i < per; ++i) {
    const int m = tid * per + i;
    if (m >= a.M) break;
    if (cta == 0 && bad_member(a, m)) ls_report(a.err, LS_DEVERR_CHECK);
    const int32_t c = drafted_of(a, m);
    tokens += c;
    units += member_units(a, m, c);
  }
  int32_t ts = tokens, us = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t x = __shfl_up_sync(0xffffffffu, ts, o), y = __shfl_up_sync(0xffffffffu, us, o);
    if (lane >= o) {
      ts += x;
      us += y;
    }
  }
  if (lane == 31) {
    scratch[warp] = ts;
    scratch[kWarps + warp] = us;
  }
  if (tid == 0) v->best = ~0ull;
  __syncthreads();
  int32_t all_tokens = 0, all_units = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const int32_t x = scratch[i], y = scratch[kWarps + i];
    if (i < warp) {
      ts += x;
      us += y;
    }
    all_tokens += x;
    all_units += y;
  }
  int32_t before = ts - tokens;
  for (int i = 0; i < per; ++i) {
    const int m = tid * per + i;
    if (m >= a.M) break;
    tok[m] = (uint16_t)before;
    if (cta == 0) out->tok[m] = before;
    before += drafted_of(a, m);
  }
  if (tid == 0) tok[a.M] = (uint16_t)all_tokens;
  // ---- how many CTAs take the prompt, in how many rounds of how long strips
  const int32_t np = (all_tokens * a.g + kPair - 1) / kPair, per_strip = np * a.hkv, ctas = a.cols;
  const bool prompt = np > 0 && a.nt > 0;
  const int32_t most = all_units > 0 ? ctas - 1 : ctas;
  auto strip_of = [&](int32_t cp, int32_t rounds) {  // tiles of a strip
    const int32_t s = min(a.nt, max(1, rounds * cp / per_strip));
    return (a.nt + s - 1) / s;
  };
  if (prompt) {
    unsigned long long best = ~0ull;
    for (int i = tid; i < most * kRounds; i += kThreads) {
      const int32_t cp = 1 + i / kRounds, strip = strip_of(cp, 1 + i % kRounds);
      const uint32_t strips = (uint32_t)(a.nt + strip - 1) / strip;
      const unsigned long long tp = (unsigned long long)((strips * per_strip + cp - 1) / cp) * (strip + kSegTiles);
      const unsigned long long tr = all_units > 0 ? (uint32_t)(all_units + ctas - cp - 1) / (ctas - cp) : 0;
      const unsigned long long x = (tp > tr ? tp : tr) << 16 | i;
      best = x < best ? x : best;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long x = __shfl_xor_sync(0xffffffffu, best, o);
      best = x < best ? x : best;
    }
    if (lane == 0) atomicMin(&v->best, best);
  }
  __syncthreads();
  const int32_t pick = prompt ? (int32_t)(v->best & 0xffff) : 0;
  const int32_t cp = prompt ? 1 + pick / kRounds : 0;
  if (tid == 0) {
    Plan& p = v->plan;
    p.tokens = all_tokens;
    p.np = np;
    p.cp = cp;
    p.strip = prompt ? strip_of(cp, 1 + pick % kRounds) : 1;
    p.strips = prompt ? (a.nt + p.strip - 1) / p.strip : 0;
    p.units = all_units;
    p.rcs = min(ctas - cp, all_units);
    p.m0 = p.off0 = 0;
    if (cta == 0) out->plan = p;
  }
  __syncthreads();
  const int32_t rcs = min(ctas - cp, all_units);
  if (cta >= cp && cta - cp < rcs) {  // the member that the first unit lies with
    const int32_t r0 = unit_bound(all_units, cta - cp, rcs);
    int32_t pre = us - units;
    if (pre <= r0 && r0 < us)
      for (int i = 0; i < per; ++i) {
        const int32_t m = tid * per + i, x = member_units(a, m, drafted_of(a, m));
        if (r0 < pre + x) {
          v->plan.m0 = m;
          v->plan.off0 = r0 - pre;
          break;
        }
        pre += x;
      }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
tree_attn_kernel(const __grid_constant__ TmapSet tm, const __grid_constant__ LsDecodeArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023) {  // the swizzled tiles' alignment, which the declaration asks for
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) ls_report(a.err, LS_DEVERR_CHECK);
    return;
  }
  Vars* vars = reinterpret_cast<Vars*>(smem + kOffVars);
  uint16_t* tok = reinterpret_cast<uint16_t*>(smem + kOffTok);
  volatile int* abort_flag = &vars->abort;
  const volatile Plan& plan = vars->plan;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t cta = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar_addr(sbase, B_KV_FULL + i), 1);
      mbar_init(bar_addr(sbase, B_KV_EMPTY + i), 2);  // one commit per issuer
      mbar_init(bar_addr(sbase, B_AUX + i), 1);
    }
    mbar_init(bar_addr(sbase, B_S_ALONE), 4);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_addr(sbase, B_Q_FULL + t), 4);
      mbar_init(bar_addr(sbase, B_S_FULL + t), 1);
      mbar_init(bar_addr(sbase, B_S_TAKEN + t), 4);  // a warp each
      mbar_init(bar_addr(sbase, B_P_FULL + t), 4);
      mbar_init(bar_addr(sbase, B_O_DONE + t), 1);
      mbar_init(bar_addr(sbase, B_DONE + t), 1);
      mbar_init(bar_addr(sbase, B_PV_DONE + t), 1);
    }
    vars->abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&vars->tmem), 512);
    tmem_relinquish();
  }
  // what the stream did before: lengths, drafts, queries and pages come from it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the combine may be launched: its blocks wait for this grid before they read from it
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  make_plan(a, vars, tok, reinterpret_cast<int32_t*>(smem + kOffRing), cta);
  fence_proxy_async_smem();  // the scratch above, before TMA writes the ring
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&vars->tmem);

  auto fail = [&](void) {
    ls_report(a.err, LS_DEVERR_TIMEOUT);
    *abort_flag = 1;
  };
  Walk walk(a, plan, tok, cta);
  Seg s;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0) {
      // ---------------------------------------------------------- K and V loads
      if (lane == 0) {
        tma_prefetch_desc(&tm.kp);
        tma_prefetch_desc(&tm.vp);
        tma_prefetch_desc(&tm.kr);
        tma_prefetch_desc(&tm.vr);
      }
      RingPos<kStages> ring;
      uint32_t fills = 0;
      Pages ld;
      bool ok = true;
      while (ok && walk.next(&s, cta)) {
        ld.open(a, s, lane);
        for (int32_t j = 0; ok && j < s.count; ++j) {
          const bool ragged = s.len - (s.key0 + j * kTile) < kTile;
          for (int kv = 0; kv < 2; ++kv) {
            ok = __all_sync(0xffffffffu, wait_bar(bar_addr(sbase, B_KV_EMPTY + ring.stage), ring.phase ^ 1) && !*abort_flag);
            if (!ok) {
              fail();
              break;
            }
            ld.issue(kv ? (s.resp ? &tm.vr : &tm.vp) : (s.resp ? &tm.kr : &tm.kp), s.kvh,
                     sbase + kOffRing + ring.stage * kTileBytes,
                     bar_addr(sbase, (kv && ragged ? B_AUX : B_KV_FULL) + ring.stage), lane, a.err);
            ring.advance();
            ++fills;
          }
          ld.advance(j + 1 < s.count, lane);
        }
      }
      // Do not leave while loads into this CTA's shared memory may still be in flight.
      for (uint32_t i = fills > kStages ? fills - kStages : 0; i < fills; ++i)
        mbar_wait(bar_addr(sbase, B_KV_FULL + i % kStages), (i / kStages) & 1);
    } else if (warp == 3) {
      // ---------------------------------------------------------- V tails
      uint32_t ring = 0, aux_phase = 0;
      bool ok = true;
      while (ok && walk.next(&s, cta)) {
        const int32_t left = s.len - (s.key0 + (s.count - 1) * kTile);
        ring += 2 * s.count;
        if (left >= kTile) continue;
        // the segment's last tile passes its source's end
        const uint32_t st = (ring - 1) % kStages;
        ok = wait_bar(bar_addr(sbase, B_AUX + st), (aux_phase >> st) & 1);
        if (!ok) break;
        aux_phase ^= 1u << st;
        uint8_t* vb = smem + kOffRing + st * kTileBytes;
        for (int i = left * 8 + lane; i < kTile * 8; i += 32) {  // row i / 8
          uint8_t* at = vb + (i >> 6) * kGroup + (i & 63) * 16;
          *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(at + kGroupHalf) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_addr(sbase, B_KV_FULL + st));
      }
      if (!ok) fail();
    } else if (lane == 0) {
      // ---------------------------------------------------------- MMA issuers
      const int t = warp - 1;
      const uint32_t idS = idesc_bf16_f32(kTile, kTile, false);
      const uint32_t idPV = idesc_bf16_f32(kTile, kD, true);
      const uint32_t dq = sdesc_lo(sbase + kOffQ + t * kTileBytes, 16);
      const uint32_t dk = sdesc_lo(sbase + kOffRing, 16);
      const uint32_t dv = sdesc_lo(sbase + kOffRing, kGroupHalf);
      const uint32_t d_s = tmem, d_p = tmem + kColP + t * (kTile / 2), d_o = tmem + kColO + t * kTile;
      auto issue_s = [&](uint32_t st) {
        const uint32_t b0 = dk + ((st * kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk & 3) * 32;
          mma_ss_groups(d_s, dq + (((kk >> 2) * kHalfBytes + off) >> 4),
                        b0 + (((kk >> 2) * kGroupHalf + off) >> 4), idS, kk > 0);
        }
      };
      auto issue_pv = [&](uint32_t st, bool accumulate) {
        const uint32_t b0 = dv + ((st * kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_groups(d_o, d_p + kk * 8, b0 + ((kk * 2 * kGroup) >> 4), idPV, (accumulate || kk > 0) ? 1u : 0u);
      };
      uint32_t seen = 0;
      RingPos<kStages> sp;
      // ring: loads before the segment; segs: segments that this tile has rows in; kc: its key tiles
      // so far; both, alone: those of segments with two row tiles and with one
      uint32_t ring = 0, segs = 0, kc = 0, both = 0, alone = 0;
      bool ok = true;
      while (ok && walk.next(&s, cta)) {
        const bool two = s.two(), mine = two || t == 0;
        const uint32_t last = ring + 2 * s.count - 1;
        // Loads are waited for in order and without gaps, and a stage is free after an arrival of
        // either issuer: behind its products, or, from the issuer of a tile without rows, as soon
        // as the load was seen.  So a stage's parity always names one fill.
        auto need = [&](uint32_t i) {
          for (; seen <= i; ++seen, sp.advance()) {
            if (!wait_bar(bar_addr(sbase, B_KV_FULL + sp.stage), sp.phase)) return false;
            if (!mine) mbar_arrive(bar_addr(sbase, B_KV_EMPTY + sp.stage));
          }
          return true;
        };
        if (!mine) {
          ok = need(last) && !*abort_flag;
          ring = last + 1;
          alone += s.count;
          continue;
        }
        ok = wait_bar(bar_addr(sbase, B_Q_FULL + t), segs & 1) && !*abort_flag;
        ++segs;
        // The tiles take the one S buffer in turn, A before B.  (Of the barriers below none is
        // ever more than a phase ahead of the one that is waited for.)
        auto s_free = [&](int32_t j) {
          if (t == 1) return wait_bar(bar_addr(sbase, B_S_TAKEN), (both + j) & 1);
          bool r = true;
          if (two ? both + j > 0 : both > 0 && j == 0)
            r = wait_bar(bar_addr(sbase, B_S_TAKEN + 1), (both + (two ? j : 0) - 1) & 1);
          if (two ? alone > 0 && j == 0 : alone + j > 0)
            r = r && wait_bar(bar_addr(sbase, B_S_ALONE), (alone + (two ? 0 : j) - 1) & 1);
          return r;
        };
        for (int32_t j = 0; ok && j <= s.count; ++j) {
          if (j < s.count) {  // S of step j goes before P V of step j - 1
            const uint32_t ki = ring + 2 * j;
            ok = need(ki) && s_free(j);
            if (!ok || *abort_flag) break;
            tc_fence_after();
            issue_s(ki % kStages);
            mma_commit(bar_addr(sbase, B_S_FULL + t));
            mma_commit(bar_addr(sbase, B_KV_EMPTY + ki % kStages));
          }
          if (j > 0) {
            const uint32_t vi = ring + 2 * j - 1;
            ok = need(vi) && wait_bar(bar_addr(sbase, B_P_FULL + t), kc & 1);
            if (!ok || *abort_flag) break;
            ++kc;
            tc_fence_after();
            issue_pv(vi % kStages, j > 1);
            mma_commit(bar_addr(sbase, B_PV_DONE + t));
            if (j == s.count) mma_commit(bar_addr(sbase, B_O_DONE + t));
            mma_commit(bar_addr(sbase, B_KV_EMPTY + vi % kStages));
          }
        }
        if (*abort_flag) break;
        ring = last + 1;
        (two ? both : alone) += s.count;
      }
      if (!ok) fail();
      // every MMA this thread issued has finished before tensor memory is released
      mma_commit(bar_addr(sbase, B_DONE + t));
      mbar_wait(bar_addr(sbase, B_DONE + t), 0);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------ softmax warpgroups
    const int t = (warp - 4) >> 2;  // tile A (0) or B (1)
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t s_col = tmem + lane_off, p_col = tmem + lane_off + kColP + t * (kTile / 2);
    const uint32_t o_col = tmem + lane_off + kColO + t * kTile;
    const float c = a.scale_log2;
    auto signal = [&](int bar) {  // by this warp
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_addr(sbase, bar));
    };
    // The next segment that this tile has rows in.
    auto next = [&]() {
      while (walk.next(&s, cta))
        if (s.rows > t * kTile) return true;
      return false;
    };
    // This warp's Q rows of segment s, into the operand layout (128-byte swizzle: chunk c of row r
    // lies at chunk c ^ (r & 7)).  Rows behind the segment's keep what was there: a row of S, P and
    // O depends on its own row of Q only, and theirs are not written out.
    auto load_q = [&]() {
      const int r0 = quad * 32, rows = s.rows - t * kTile;
      if (r0 >= rows) return;
      const int32_t x = s.row0 + t * kTile + min(r0 + lane, rows - 1), at = x / a.g, head = x - at * a.g;
      int32_t m = s.m, first = at;  // member, and the token among its drafted ones
      if (!s.resp) {
        int32_t lo = 0, hi = a.M - 1;  // the last member whose tokens begin at or before `at`
        while (lo < hi) {
          const int32_t mid = (lo + hi + 1) >> 1;
          if (tok[mid] <= at) lo = mid; else hi = mid - 1;
        }
        m = lo;
        first = at - tok[lo];
      }
      const int32_t src = (m * a.n + a.n - (tok[m + 1] - tok[m]) + first) * a.hq + s.kvh * a.g + head;
      const int c = lane & 15;
      const uint32_t dst = sbase + kOffQ + t * kTileBytes + (c >> 3) * kHalfBytes;
#pragma unroll 8
      for (int k = 0; k < 16; ++k) {
        const int r = r0 + 2 * k + (lane >> 4);
        const int32_t from = __shfl_sync(0xffffffffu, src, 2 * k + (lane >> 4));
        if (r < rows)
          cp_async16(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                     static_cast<const __nv_bfloat16*>(a.q) + (int64_t)from * kD + c * 8);
      }
    };
    auto q_loaded = [&]() {
      cp_async_wait_all();
      fence_proxy_async_smem();
      signal(B_Q_FULL + t);
    };
    uint32_t kc = 0, oc = 0;
    bool ok = true, have = next();
    if (have) {
      load_q();
      q_loaded();
    }
    while (ok && have) {
      const int32_t rows = s.rows - t * kTile;  // of this tile
      const int taken = s.two() ? B_S_TAKEN + t : B_S_ALONE;
      const bool idle = quad * 32 >= rows;  // the whole warp is padding
      // keys from its first key tile on that every row sees: the source's, or the context
      int32_t lim = s.len - s.key0, pad = 0;
      const uint32_t* bits = nullptr;
      if (s.resp) {
        const int32_t drafted = tok[s.m + 1] - tok[s.m];
        pad = a.n - drafted;
        lim -= drafted;
        const int32_t at = min(s.row0 + t * kTile + row, s.row0 + s.rows - 1) / a.g;
        bits = a.visible + ((int64_t)s.m * a.n + pad + at) * a.words;
      }
      float m = -INFINITY, l = 0.f, lcomp = 0.f;
      for (int32_t j = 0; j < s.count; ++j, ++kc, lim -= kTile) {
        ok = wait_bar(bar_addr(sbase, B_S_FULL + t), kc & 1);
        if (!ok) break;
        // P's columns are free, and O may be changed, after P V of the tile before.
        auto settled = [&]() { return j == 0 || wait_bar(bar_addr(sbase, B_PV_DONE + t), (kc - 1) & 1); };
        if (idle) {  // P keeps what was there: rows of D depend on their own rows of A only
          signal(taken);
          ok = settled();
          if (!ok) break;
          signal(B_P_FULL + t);
          continue;
        }
        tc_fence_after();
        uint32_t sr[128];
        tmem_ld32(s_col + 0, sr);
        tmem_ld32(s_col + 32, sr + 32);
        tmem_ld32(s_col + 64, sr + 64);
        tmem_ld32(s_col + 96, sr + 96);
        tmem_wait_ld();
        reg_fence32(sr);
        reg_fence32(sr + 32);
        reg_fence32(sr + 64);
        reg_fence32(sr + 96);
        signal(taken);
        if (lim < kTile) {
          if (s.resp) {  // drafted keys among these
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint64_t see = tree_window(a, bits, pad - lim + 64 * hf, pad);
#pragma unroll
              for (int e = 0; e < 64; ++e)
                if (!((uint32_t)(see >> (e & 32)) & (1u << (e & 31)))) sr[64 * hf + e] = __float_as_uint(-INFINITY);
            }
          } else {  // the prompt's ragged end
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (e >= lim) sr[e] = __float_as_uint(-INFINITY);
          }
        }
        float mx8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(__uint_as_float(sr[k]), __uint_as_float(sr[k + 8]));
#pragma unroll
        for (int e = 16; e < 128; e += 16)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mx8[k] = fmax3(mx8[k], __uint_as_float(sr[e + k]), __uint_as_float(sr[e + 8 + k]));
        const float mt = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                               fmaxf(mx8[6], mx8[7])) * c;
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
        // rescale O first (rare): P_t V of this tile adds to it as soon as the first half of P
        // is in tensor memory
        if (__any_sync(0xffffffffu, rescale)) {
          ok = settled();
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 0; c0 < kD; c0 += 32) {
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
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // P in two halves of 64 keys
          uint32_t pk[32];
#pragma unroll
          for (int jj = 0; jj < 32; ++jj) {
            const int e = half * 32 + jj;
            float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1])),
                                  c2, nm2);
            x.x = fast_exp2(x.x);
            x.y = fast_exp2(x.y);
            ls4[jj & 3] = __fadd2_rn(ls4[jj & 3], x);
            // weights in [0, 2^8] enter the product as bf16, as in the replay forward: their
            // roundings are independent, so o's error is that of one bf16 rounding
            pk[jj] = pack_bf16(x.x, x.y);
          }
          if (half == 0) {
            ok = settled();
            if (!ok) break;
            tc_fence_after();
          }
          tmem_st32(p_col + half * 32, pk);
        }
        if (!ok) break;
        tmem_wait_st();
        signal(B_P_FULL + t);
        const float2 lsa = __fadd2_rn(__fadd2_rn(ls4[0], ls4[1]), __fadd2_rn(ls4[2], ls4[3]));
        const float ls = lsa.x + lsa.y;
        const float tsum = l + ls;
        lcomp += (l - tsum) + ls;
        l = tsum;
      }
      if (!ok) break;
      // the next segment's Q rows (this one's last S is done), while P V is
      const int64_t prow = s.part + t * kTile + row;
      if (tid == 128 && s.resp) {
        int32_t* range = cta_range(a, s.m, s.row0 / kPair, s.kvh);
        if (s.key0 == 0) range[0] = cta - plan.cp;
        if (s.len - s.key0 <= s.count * kTile) range[1] = cta - plan.cp;
      }
      have = next();
      if (have) load_q();
      ok = wait_bar(bar_addr(sbase, B_O_DONE + t), oc & 1);
      if (!ok) break;
      ++oc;
      if (have) q_loaded();
      if (!idle) {
        tc_fence_after();
        const float lt = l + lcomp;
        const float inv = lt == 0.f ? 0.f : 1.f / lt;  // a row that sees no key here
        float* po = part_at(a, prow);
#pragma unroll 1
        for (int c0 = 0; c0 < kD; c0 += 32) {
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
        if (row < rows) a.part_lse[prow] = lt == 0.f ? -INFINITY : m + log2f(lt);
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
// order.  Eight drafted rows of one member and KV head are a block's, a thread four values of one of
// them, or (kWide) a warp's, a thread 32 values; a warp's loads are whole lines of the partials (eight
// rows, four values of each in turn).  With many rows there are few partials of each, and what a
// thread does besides its values counts (2,784 tokens of 16 / 8 heads over 46 and responses of up to
// 464: the call takes 87 us with a block, 64 with a warp); with few rows there are many, and the loads
// under way count.
constexpr int kCombineWarps = 8;

template <bool kWide>
__global__ void __launch_bounds__(kCombineWarps * 32)
tree_combine(const __grid_constant__ LsDecodeArgs a) {
  constexpr int kChunks = kWide ? 8 : 1, kBatch = kWide ? 2 : 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t octets = (a.n * a.g + 7) >> 3, blocks = kWide ? (octets + 7) >> 3 : octets;
  const int32_t m = blockIdx.x / blocks, h = blockIdx.y, b = blockIdx.x - m * blocks;
  const int32_t tokens = drafted_of(a, m);
  const int32_t chunk = (kWide ? 0 : warp * 4) + (lane >> 3);                    // the first; then every fourth
  const int32_t mrow = 8 * (kWide ? b * 8 + warp : b) + (lane & 7);  // among the drafted ones
  const bool resp = clamp_len(a, __ldg(a.lens + m)) > 0;
  // Rows that are not written (padding, members out of use) wait all the same: the stream goes
  // on when this grid ends.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (mrow >= tokens * a.g) return;
  const Out* out = static_cast<const Out*>(a.plan);
  const int32_t rpair = mrow / kPair;
  const int32_t* range = cta_range(a, m, rpair, h);
  const int32_t np = __ldcg(&out->plan.np), strips = __ldcg(&out->plan.strips);
  const int32_t prow = __ldcg(out->tok + m) * a.g + mrow, pair = prow / kPair;
  const int32_t rc = resp ? __ldcg(range) : 0, segs = resp ? __ldcg(range + 1) + 1 - rc : 0;
  const int64_t prompt0 = (int64_t)(h * strips * np + pair) * kPair + (prow - pair * kPair);
  const int64_t resp0 = resp_row0(a, m, rpair, h, rc) + (mrow - rpair * kPair);
  const int32_t count = strips + segs;
  auto part_row = [&](int32_t k) {
    return k < strips ? prompt0 + (int64_t)k * np * kPair
                      : resp0 + (int64_t)(k - strips) * resp_rows_of(a);
  };
  float mx = -INFINITY, sum = 0.f;
  float4 acc[kChunks];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int32_t k0 = 0; k0 < count; k0 += kBatch) {
    float l[kBatch];
    float4 v[kBatch][kChunks];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      l[k] = -INFINITY;
      if (k0 + k < count) {
        const int64_t r = part_row(k0 + k);
        l[k] = __ldcg(a.part_lse + r);
        const float* p = part_at(a, r) + chunk * 32;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) v[k][c] = __ldcg(reinterpret_cast<const float4*>(p + c * 128));
      }
    }
    float top = mx;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) top = fmaxf(top, l[k]);
    if (top == -INFINITY) continue;
    const float old = exp2f(mx - top);
    mx = top;
    sum *= old;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      acc[c] = make_float4(acc[c].x * old, acc[c].y * old, acc[c].z * old, acc[c].w * old);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (l[k] == -INFINITY) continue;  // a part that saw no key adds nothing
      const float w = exp2f(l[k] - mx);
      sum += w;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        acc[c].x = fmaf(w, v[k][c].x, acc[c].x);
        acc[c].y = fmaf(w, v[k][c].y, acc[c].y);
        acc[c].z = fmaf(w, v[k][c].z, acc[c].z);
        acc[c].w = fmaf(w, v[k][c].w, acc[c].w);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key at all: o = 0, lse = -inf
  const int32_t row = (a.n - tokens) * a.g + mrow;  // the drafted ones are the member's last
  const int64_t to = ((int64_t)m * a.n + row / a.g) * a.hq + h * a.g + row % a.g;
  __nv_bfloat16* po = static_cast<__nv_bfloat16*>(a.o) + to * kD + chunk * 4;
#pragma unroll
  for (int c = 0; c < kChunks; ++c)
    *reinterpret_cast<uint2*>(po + c * 16) = make_uint2(pack_bf16(acc[c].x * inv, acc[c].y * inv),
                                                        pack_bf16(acc[c].z * inv, acc[c].w * inv));
  if (chunk == 0) a.lse[to] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
}

}  // namespace

size_t ls_tree_plan_bytes(const LsDecodeArgs& a) {
  return sizeof(Out) + (size_t)a.M * max_pairs(a) * a.hkv * 2 * sizeof(int32_t);
}
int64_t ls_tree_part_rows(const LsDecodeArgs& a) {
  const int64_t slots = (int64_t)a.M * max_pairs(a) * a.hkv + a.cols;
  return prompt_rows_of(a) + slots * resp_rows_of(a);
}

cudaError_t ls_launch_tree_attn(const LsDecodeArgs& a, cudaStream_t st) {
  TmapSet tm;
  if (!make_tmaps(a, &tm, true)) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.cols);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, tree_attn_kernel, tm, a)) != cudaSuccess) return e;
  ls_note_launch();
  cfg.dynamicSmemBytes = 0;
  // rows enough for a warp an SM and four schedulers
  const int octets = (a.n * a.g + 7) / 8;
  const bool wide = (int64_t)a.M * octets * a.hkv >= 8 * a.cols;
  cfg.gridDim = dim3((unsigned)(a.M * (wide ? (octets + 7) / 8 : octets)), (unsigned)a.hkv);
  cfg.blockDim = dim3(kCombineWarps * 32);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = wide ? cudaLaunchKernelEx(&cfg, tree_combine<true>, a) : cudaLaunchKernelEx(&cfg, tree_combine<false>, a);
  if (e == cudaSuccess) ls_note_launch();
  return e;
}
