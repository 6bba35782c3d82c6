// ls_decode.cuh -- what the kernels of a decode step share (decode_attn.cu, tree_attn.cu): tiles
// of keys and values gathered page by page, the layout of partial results, and what a row of a
// drafted tree sees.
#pragma once
#include <math.h>

#include "ls_device.cuh"
#include "ls_internal.h"
#include "ls_tmap.h"
#include "ls_umma.cuh"

namespace decode {

using namespace umma;

constexpr int kD = 128;
constexpr int kTile = 128;  // keys, and query rows, of a tile
constexpr uint32_t kTileBytes = kTile * kD * 2;
constexpr uint32_t kHalfBytes = kTileBytes / 2;
constexpr int kMaxBoxes = kTile / 16;  // a tile's pages at the smallest page size
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;

struct TmapSet {
  CUtensorMap kp, vp, kr, vr;
};

// A bounded wait that asks once without the suspend: most of the issuing warps' waits find
// their phase complete.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity) {
  return mbar_try_wait(bar, parity) || mbar_wait(bar, parity);
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// A member's response keys: none for a member out of use (negative length); a length
// past its row of the block table is cut (and reported by the main kernel).
__device__ __forceinline__ int32_t clamp_len(const LsDecodeArgs& a, int32_t len) {
  const long long room = (long long)a.max_blocks << a.r_ps_log2;
  if (len < 0) return 0;
  return len < room ? len : (int32_t)room;
}
__device__ __forceinline__ int32_t tiles_of(int32_t len) {
  return (int32_t)(((long long)len + kTile - 1) / kTile);
}
// Drafted tokens of a member, the last of its n: a count outside 0 .. min(n, its length) is cut (and
// reported by the main kernel).
__device__ __forceinline__ int32_t drafted_of(const LsDecodeArgs& a, int32_t m) {
  const int32_t len = __ldg(a.lens + m), c = a.drafted ? __ldg(a.drafted + m) : a.n;
  return max(min(c, min(a.n, len)), 0);
}
// Whether a member's length and draft are not what they may be.
__device__ __forceinline__ bool bad_member(const LsDecodeArgs& a, int32_t m) {
  const int32_t len = __ldg(a.lens + m);
  if (len > clamp_len(a, len)) return true;
  const int32_t c = a.drafted ? __ldg(a.drafted + m) : a.n;
  return len >= 0 && (c < 0 || c > a.n || c > len);
}

// What a row of a tree may see of the 64 keys from key kb on: the member's context (the keys
// before its drafted ones), and of the drafted ones those of its bits.  d: kb counted from the
// key of the member's first row; pad: rows before the first drafted one.
__device__ __forceinline__ uint64_t tree_window(const LsDecodeArgs& a, const uint32_t* bits, int32_t d,
                                                int32_t pad) {
  auto words = [&](int32_t at) {  // bits 32 at .. 32 at + 31 of the row
    const int32_t lo = pad - 32 * at, hi = a.n - 32 * at;
    uint32_t x = at >= 0 && at < a.words ? __ldg(bits + at) : 0u;
    if (hi < 32) x &= hi > 0 ? (1u << hi) - 1 : 0u;
    if (lo > 0) x |= lo < 32 ? (1u << lo) - 1 : 0xffffffffu;
    return x;
  };
  const int32_t at = d >> 5, sh = d & 31;
  const uint32_t w0 = words(at), w1 = words(at + 1), w2 = words(at + 2);
  return (uint64_t)__funnelshift_r(w0, w1, sh) | (uint64_t)__funnelshift_r(w1, w2, sh) << 32;
}

// The loads of one ring (K or V) of a CTA, issued by one thread.  A tile's pages are looked
// up while the last tile's loads are under way.  Whole-tile boxes (pages of 128 rows and
// more) come with both 64-dim halves in one copy; smaller pages take two copies a page.
struct Loader {
  const void* map;              // of the segment's source
  const int32_t* table;
  int32_t len, key0, boxes, box_rows, ps_log2, pages, hkv, kvh, pool_rows;
  int32_t page[kMaxBoxes];

  // resp, m: whether a response's keys, and whose; head_: KV head; from key first on of n
  __device__ __forceinline__ void open(const LsDecodeArgs& a, bool resp, int32_t m, int32_t head_,
                                       int32_t first, int32_t n, const void* prompt_map,
                                       const void* resp_map) {
    map = resp ? resp_map : prompt_map;
    table = resp ? a.blocks + (int64_t)m * a.max_blocks : a.page_table;
    ps_log2 = resp ? a.r_ps_log2 : a.ps_log2;
    pages = resp ? a.r_num_pages : a.num_pages;
    box_rows = min(1 << ps_log2, kTile);
    boxes = kTile / box_rows;
    pool_rows = (pages * a.hkv) << ps_log2;
    hkv = a.hkv;
    kvh = head_;
    len = n;
    key0 = first;
    look_up();
  }
  __device__ __forceinline__ void look_up() {
#pragma unroll
    for (int x = 0; x < kMaxBoxes; ++x)
      if (x < boxes && key0 + x * box_rows < len) page[x] = __ldg(table + ((key0 + x * box_rows) >> ps_log2));
  }
  // one tile to `dst`, counted on barrier `bar`; then the next tile's pages
  __device__ __forceinline__ void load(uint32_t dst, uint32_t bar, bool more, uint32_t* err) {
    mbar_expect_tx(bar, kTileBytes);
#pragma unroll
    for (int x = 0; x < kMaxBoxes; ++x) {
      if (x >= boxes) break;
      int32_t y = pool_rows;  // out of bounds: zero fill
      if (key0 + x * box_rows < len) {
        if ((uint32_t)page[x] < (uint32_t)pages)
          y = ((page[x] * hkv + kvh) << ps_log2) + ((key0 + x * box_rows) & ((1 << ps_log2) - 1));
        else
          ls_report(err, LS_DEVERR_CHECK);
      }
      if (boxes == 1) {
        tma_load_3d(dst, map, 0, y, 0, bar);
      } else {
        tma_load_2d(dst + x * box_rows * 128, map, 0, y, bar);
        tma_load_2d(dst + kHalfBytes + x * box_rows * 128, map, 64, y, bar);
      }
    }
    key0 += kTile;
    if (more) look_up();
  }
};

// Rows of partial results lie in eights, four values of each in turn (see decode_attn.cu).
__device__ __forceinline__ float* part_at(const LsDecodeArgs& a, int64_t row) {
  return a.part_o + (row >> 3) * (8 * kD) + (row & 7) * 4;  // values 4 c .. 4 c + 3 at 32 c
}

// Tensor maps of the prompt's and the responses' pools: rows of 256 bytes; a whole-tile box
// takes both halves of its rows, half by half.
// Grouped: boxes are [eight rows][half][row][64 values], so a box of any height is one copy and a
// tile's groups of eight rows lie 2 KB apart, their halves 1 KB.
inline bool make_tmaps(const LsDecodeArgs& a, TmapSet* tm, bool grouped = false) {
  for (int src = 0; src < 2; ++src) {
    const int ps = 1 << (src ? a.r_ps_log2 : a.ps_log2);
    const uint64_t rows = (uint64_t)(src ? a.r_num_pages : a.num_pages) * a.hkv * ps;
    const bool whole = ps >= kTile;
    const uint64_t dims[3] = {whole ? 64u : (uint64_t)kD, rows, 2};
    const uint64_t strides[2] = {(uint64_t)kD * 2, (uint64_t)kD};
    const uint32_t box[3] = {64, (uint32_t)(ps < kTile ? ps : kTile), 2};
    const int rank = whole ? 3 : 2;
    if (grouped) {
      const uint64_t gdims[4] = {64, 8, 2, rows / 8}, gstrides[3] = {(uint64_t)kD * 2, (uint64_t)kD, (uint64_t)kD * 16};
      const uint32_t gbox[4] = {64, 8, 2, box[1] / 8};
      if (!ls_make_tmap_bf16(src ? &tm->kr : &tm->kp, src ? a.rk_pool : a.k_pool, 4, gdims, gstrides, gbox) ||
          !ls_make_tmap_bf16(src ? &tm->vr : &tm->vp, src ? a.rv_pool : a.v_pool, 4, gdims, gstrides, gbox))
        return false;
      continue;
    }
    if (!ls_make_tmap_bf16(src ? &tm->kr : &tm->kp, src ? a.rk_pool : a.k_pool, rank, dims, strides, box) ||
        !ls_make_tmap_bf16(src ? &tm->vr : &tm->vp, src ? a.rv_pool : a.v_pool, rank, dims, strides, box))
      return false;
  }
  return true;
}

}  // namespace decode
