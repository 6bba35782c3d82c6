// drafts.cu -- trees of drafted tokens: what a node sees, which path the policy accepts, and
// the moves of accepted keys and values (and of whole pages) in every layer's pages.
//
// A member's draft is the last `drafted` of its n rows; row r's node continues row
// parents[r] < r of the same draft, or (-1) the member's context.  Node r sees itself and its
// ancestors: with anc(r) a row's ancestor and see(r) the rows known to be seen from it,
//   see(r) |= see(anc(r)),  anc(r) = anc(anc(r))
// doubles the known part of every path, so log2(depth) + 1 rounds reach every root.  The accepted path
// is the same doubling over "the policy chose this node after its parent".
//
// Both are one block a member and bound by a launch and these rounds.
// The moves are bound by HBM, or, at a decode step's few rows, by a launch and two dependent
// loads (rows, pages) in front of the copies.
#include "ls_device.cuh"
#include "ls_internal.h"

namespace {

constexpr int kMaxRows = 128;
constexpr int kWords = kMaxRows / 32;

struct Member {
  int len, drafted, first;  // first: the first drafted row; n for a member out of use
};
__device__ __forceinline__ Member member_of(const LsDraftArgs& a, int m, bool report) {
  Member x;
  x.len = __ldg(a.lens + m);
  x.drafted = a.drafted ? __ldg(a.drafted + m) : a.n;
  if (x.len < 0) {
    x.drafted = 0;
  } else if (x.drafted < 0 || x.drafted > a.n || x.drafted > x.len) {
    if (report) ls_report(a.err, LS_DEVERR_CHECK);
    x.drafted = min(max(x.drafted, 0), min(a.n, x.len));
  }
  x.first = a.n - x.drafted;
  return x;
}
// A row's parent, or -1; one outside its draft's earlier rows is refused and taken as -1.
__device__ __forceinline__ int parent_of(const LsDraftArgs& a, int m, int r, const Member& x) {
  const int p = __ldg(a.parents + (int64_t)m * a.n + r);
  if (p >= x.first && p < r) return p;
  if (p != -1) ls_report(a.err, LS_DEVERR_CHECK);
  return -1;
}

__global__ void __launch_bounds__(kMaxRows) draft_tree_kernel(const LsDraftArgs a, uint32_t* visible,
                                                              int32_t* positions, int axes, int pos0) {
  __shared__ uint32_t see[kMaxRows][kWords + 1];  // a column apart: rows meet other banks
  __shared__ int anc[kMaxRows];
  const int m = blockIdx.x, r = threadIdx.x;
  const Member x = member_of(a, m, r == 0);
  const bool real = r < a.n && r >= x.first;
  uint32_t mine[kWords];
#pragma unroll
  for (int w = 0; w < kWords; ++w) mine[w] = real && w == (r >> 5) ? 1u << (r & 31) : 0u;
  int up = real ? parent_of(a, m, r, x) : -1;
  anc[r] = up;
#pragma unroll
  for (int w = 0; w < kWords; ++w) see[r][w] = mine[w];
  while (__syncthreads_or(up >= 0)) {
    int next = -1;
    if (up >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) mine[w] |= see[up][w];
      next = anc[up];
    }
    __syncthreads();
    if (up >= 0) {
#pragma unroll
      for (int w = 0; w < kWords; ++w) see[r][w] = mine[w];
      anc[r] = next;
    }
    up = next;
  }
  if (r >= a.n) return;
  const int words = (a.n + 31) >> 5;
  uint32_t* out = visible + ((int64_t)m * a.n + r) * words;
  int depth = -1;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    depth += __popc(mine[w]);
    if (w < words) out[w] = mine[w];
  }
  if (positions) {
    const int32_t pos = real ? (int32_t)((uint32_t)pos0 + (uint32_t)(x.len - x.drafted + depth)) : 0;
    for (int i = 0; i < axes; ++i) positions[((int64_t)i * a.members + m) * a.n + r] = pos;
  }
}

__global__ void __launch_bounds__(kMaxRows) accept_draft_kernel(
    const LsDraftArgs a, const int32_t* __restrict__ tokens, const int32_t* __restrict__ chosen,
    int32_t* rows, int32_t* count, int32_t* follow, int32_t* ends) {
  __shared__ int want[kMaxRows], first_of[kMaxRows], anc[kMaxRows];
  __shared__ uint32_t kept[kWords];
  __shared__ bool ok[kMaxRows];
  const int m = blockIdx.x, r = threadIdx.x;
  const Member x = member_of(a, m, r == 0);
  const bool real = r < a.n && r >= x.first;
  const int64_t at = (int64_t)m * a.n + r;
  want[r] = real ? __ldg(chosen + at) : -1;
  first_of[r] = kMaxRows;
  int up = real ? parent_of(a, m, r, x) : -1;
  const int token = real ? __ldg(tokens + at) : -1;
  __syncthreads();
  // chosen after its parent, and the first of the parent's children that is
  const bool match = up >= 0 && token >= 0 && token == want[up];
  if (match) atomicMin(first_of + up, r);
  __syncthreads();
  bool good = real && (r == x.first || (match && first_of[up] == r));
  anc[r] = up;
  ok[r] = good;
  while (__syncthreads_or(up >= 0)) {
    int next = -1;
    if (up >= 0) {
      good = good && ok[up];
      next = anc[up];
    }
    __syncthreads();
    if (up >= 0) {
      ok[r] = good;
      anc[r] = next;
    }
    up = next;
  }
  const uint32_t mask = __ballot_sync(0xffffffffu, good);
  if ((r & 31) == 0) kept[r >> 5] = mask;
  __syncthreads();
  int n = 0, before = 0, last = -1;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    const uint32_t k = kept[w];
    if (w < (r >> 5)) before += __popc(k);
    n += __popc(k);
    if (k) last = 32 * w + 31 - __clz(k);
  }
  before += __popc(mask & ((1u << (r & 31)) - 1));
  if (good) rows[(int64_t)m * a.n + before] = r;
  if (r >= n && r < a.n) rows[at] = -1;
  if (r == 0) {
    count[m] = n;
    follow[m] = last >= 0 ? want[last] : -1;
    ends[m] = x.len < 0 ? x.len : x.len - x.drafted + n;
  }
}

// ---------------------------------------------------------------- accepted rows

constexpr int kMoveWarps = 8;

// A block moves the kept rows of one member and layer: row i of `rows` goes to the i-th key behind
// the context.  It looks the rows' places up once; then a warp takes a KV head of a pool at a time.
// Rows ascend, so i <= its row, and a key is written only after every row that could be read from
// it has been (in this batch's loads or before).  (A warp of its own a head and pool, each with
// its own look-ups: 43 us for the 202 MB of 256 members in 16 layers, now 36.)
__global__ void __launch_bounds__(kMoveWarps * 32) compact_rows_kernel(
    const LsLayerPools p, const int32_t* __restrict__ table, int max_blocks, const LsDraftArgs a,
    const int32_t* __restrict__ rows, const int32_t* __restrict__ count) {
  __shared__ int64_t from[kMaxRows], to[kMaxRows];  // in 16 bytes, under KV head 0; -1: not moved
  const int tid = threadIdx.x, lane = tid & 31, warps = blockDim.x >> 5;
  const int m = blockIdx.x, layer = blockIdx.y;
  const Member x = member_of(a, m, layer == 0 && tid == 0);
  const int n = __ldg(count + m);
  const int64_t room = (int64_t)max_blocks << p.ps_log2;
  bool bad = n < 0 || n > x.drafted || x.len > room;
  // rows of the draft, ascending: so row i is the i-th drafted one or a later one
  const int32_t* mine = rows + (int64_t)m * a.n;
  const int32_t* blocks = table + (int64_t)m * max_blocks;
  const int base = x.len - x.drafted;
  auto key_at = [&](int key, int* page) {  // of KV head 0
    *page = __ldg(blocks + (key >> p.ps_log2));
    return (((int64_t)*page * p.hkv) << p.ps_log2 | (key & ((1 << p.ps_log2) - 1))) * 16;
  };
  for (int i = tid; !bad && i < n; i += blockDim.x) {
    const int r = __ldg(mine + i), prev = i > 0 ? __ldg(mine + i - 1) : x.first - 1;
    if (r <= prev || r >= a.n) bad = true;
    if (bad) break;
    from[i] = -1;
    if (r - x.first == i) continue;
    int pf, pt;
    const int64_t f = key_at(base + r - x.first, &pf), t = key_at(base + i, &pt);
    if ((uint32_t)pf >= (uint32_t)p.num_pages || (uint32_t)pt >= (uint32_t)p.num_pages) {
      if (layer == 0) ls_report(a.err, LS_DEVERR_CHECK);
    } else {
      from[i] = f;
      to[i] = t;
    }
  }
  if (__syncthreads_or(bad)) {
    if (layer == 0 && tid == 0) ls_report(a.err, LS_DEVERR_CHECK);
    return;
  }
  constexpr int kBatch = 4;  // two rows a step
  const int half = lane >> 4, c = lane & 15;
  for (int item = tid >> 5; item < 2 * p.hkv; item += warps) {
    uint4* pool = reinterpret_cast<uint4*>(
        static_cast<__nv_bfloat16*>(item & 1 ? p.v_pool : p.k_pool) + layer * p.stride) +
        (((int64_t)(item >> 1) << p.ps_log2) * 16 + c);
    for (int i0 = 0; i0 < n; i0 += 2 * kBatch) {
      uint4 v[kBatch];
      bool moves[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = i0 + 2 * b + half;
        moves[b] = i < n && from[i] >= 0;
        if (moves[b]) v[b] = pool[from[i]];
      }
      __syncwarp();
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (moves[b]) pool[to[i0 + 2 * b + half]] = v[b];
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------- whole pages

constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 64;  // rows of a block: 16 KB

// Block (x, y): a pair of pages under one layer, KV head and pool (x); 64 of its rows (y).
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(
    const LsLayerPools p, int count, const int32_t* __restrict__ from, const int32_t* __restrict__ to,
    const int32_t* __restrict__ rows, uint32_t* err) {
  const int64_t per = (int64_t)p.layers * p.hkv * 2;
  const int i = (int)(blockIdx.x / per);
  const int64_t item = blockIdx.x - i * per;
  const int f = __ldg(from + i), t = __ldg(to + i);
  const int ps = 1 << p.ps_log2;
  int n = rows ? __ldg(rows + i) : ps;
  if (f < 0 && t < 0) return;  // nothing to copy
  if ((uint32_t)f >= (uint32_t)p.num_pages || (uint32_t)t >= (uint32_t)p.num_pages || n < 0 || n > ps) {
    if (item == 0 && blockIdx.y == 0 && threadIdx.x == 0) ls_report(err, LS_DEVERR_CHECK);
    return;
  }
  if (f == t) return;
  const int layer = (int)(item / (2 * p.hkv)), h = (int)(item >> 1) % p.hkv;
  uint4* pool = reinterpret_cast<uint4*>(
      static_cast<__nv_bfloat16*>(item & 1 ? p.v_pool : p.k_pool) + layer * p.stride);
  const int r0 = blockIdx.y * kCopyRows;
  const int vecs = (min(n - r0, kCopyRows)) * 16;
  const uint4* src = pool + ((((int64_t)f * p.hkv + h) << p.ps_log2) + r0) * 16;
  uint4* dst = pool + ((((int64_t)t * p.hkv + h) << p.ps_log2) + r0) * 16;
  constexpr int kPer = kCopyRows * 16 / kCopyThreads;
  uint4 v[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if ((int)threadIdx.x + k * kCopyThreads < vecs) v[k] = src[threadIdx.x + k * kCopyThreads];
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if ((int)threadIdx.x + k * kCopyThreads < vecs) dst[threadIdx.x + k * kCopyThreads] = v[k];
}

}  // namespace

cudaError_t ls_launch_draft_tree(const LsDraftArgs& a, int32_t* visible, int32_t* positions,
                                 int32_t axes, int32_t pos0, cudaStream_t st) {
  draft_tree_kernel<<<a.members, kMaxRows, 0, st>>>(a, reinterpret_cast<uint32_t*>(visible), positions,
                                                    axes, pos0);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ls_note_launch();
  return e;
}

cudaError_t ls_launch_accept_draft(const LsDraftArgs& a, const int32_t* tokens,
                                   const int32_t* chosen, int32_t* rows, int32_t* count,
                                   int32_t* follow, int32_t* ends, cudaStream_t st) {
  accept_draft_kernel<<<a.members, kMaxRows, 0, st>>>(a, tokens, chosen, rows, count, follow, ends);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ls_note_launch();
  return e;
}

cudaError_t ls_launch_compact_rows(const LsLayerPools& p, const int32_t* table, int32_t max_blocks,
                                   const LsDraftArgs& a, const int32_t* rows, const int32_t* count,
                                   cudaStream_t st) {
  const int warps = 2 * p.hkv < kMoveWarps ? 2 * p.hkv : kMoveWarps;
  compact_rows_kernel<<<dim3(a.members, p.layers), warps * 32, 0, st>>>(
      p, table, max_blocks, a, rows, count);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ls_note_launch();
  return e;
}

cudaError_t ls_launch_copy_pages(const LsLayerPools& p, int32_t count, const int32_t* from,
                                 const int32_t* to, const int32_t* rows, uint32_t* err,
                                 cudaStream_t st) {
  const int64_t items = (int64_t)count * p.layers * p.hkv * 2;
  const int chunks = ((1 << p.ps_log2) + kCopyRows - 1) / kCopyRows;
  copy_pages_kernel<<<dim3((unsigned)items, chunks), kCopyThreads, 0, st>>>(p, count, from, to, rows, err);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ls_note_launch();
  return e;
}
