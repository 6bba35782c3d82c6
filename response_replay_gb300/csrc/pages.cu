// pages.cu -- pages and slots of growing sequences, built on the GPU from their lengths.
//
// Member m holds lens[m] tokens in the pages of its row of the block table and is to
// hold add[m] more.  With ps the page size it owns have = ceil(len / ps) pages and needs
// ceil((len + add) / ps); the missing ones are taken from the free list in member order
// (an exclusive sum over the members gives each its first), entered into the table, and
// token i of the member gets slot table[i / ps] * ps + i % ps and position pos0 + i.
// The new tokens stand packed, member after member, or each member's as the last of its own
// `rows` rows, which is where a step of fixed rows has them whoever adds how many.
//
// Nothing here depends on another block: every block sums the members' counts itself
// (at most 1,024 members, one per thread; 8 KB from L2) and then fills its share of the
// tokens and of the new table entries, so one launch serves any length.  The lengths and
// the count of used pages are read by every block; they are written by the only block of
// a small call, by block 0 when they go to buffers of their own, and by a second launch
// when a large call writes them over what it reads.
//
// It is bound by a launch and one dependent chain (lengths, two scans, a search, a page, a
// slot): one token for each of 8 members 4.0 us, 282,000 tokens for 64 members 5.2 us, of
// which the 2.2 MB of slots and positions are 0.3 us at the copy's rate.
#include "ls_device.cuh"
#include "ls_internal.h"

namespace {

constexpr int kThreads = 1024;
constexpr int kPerThread = 4;                      // consecutive tokens of a thread
constexpr int kChunk = kThreads * kPerThread;      // tokens of a block

struct Plan {
  long long tok_end[kThreads];  // tokens up to and including the member
  int page_end[kThreads];       // new pages up to and including the member
  int len[kThreads], have[kThreads];
  int used0;
  bool ok;
};

// Inclusive sums over the block's threads, warp by warp.
__device__ __forceinline__ void block_scan(long long* tok, int* pages, long long* wt, int* wp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, *tok, o);
    const int p = __shfl_up_sync(0xffffffffu, *pages, o);
    if (lane >= o) {
      *tok += t;
      *pages += p;
    }
  }
  if (lane == 31) {
    wt[warp] = *tok;
    wp[warp] = *pages;
  }
  __syncthreads();
  if (warp == 0) {
    long long t = wt[lane];
    int p = wp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t2 = __shfl_up_sync(0xffffffffu, t, o);
      const int p2 = __shfl_up_sync(0xffffffffu, p, o);
      if (lane >= o) {
        t += t2;
        p += p2;
      }
    }
    wt[lane] = t;
    wp[lane] = p;
  }
  __syncthreads();
  if (warp > 0) {
    *tok += wt[warp - 1];
    *pages += wp[warp - 1];
  }
}

__device__ __forceinline__ int32_t page_of(const LsExtendArgs& a, const Plan& p, int m, int b) {
  if (b < p.have[m]) return a.table[(int64_t)m * a.max_blocks + b];
  const int before = m ? p.page_end[m - 1] : 0;
  return __ldg(a.free_list + p.used0 + before + b - p.have[m]);
}

// fill: slots, positions and table entries; commit: lens_out and used_out.  kRows: every
// member has rows of its own (a template, as a test of it for every token made the packed
// call 0.3 us longer).
template <bool kRows>
__global__ void __launch_bounds__(kThreads) extend_pages_kernel(const LsExtendArgs a, int fill,
                                                                int commit) {
  __shared__ Plan p;
  __shared__ long long wt[32];
  __shared__ int wp[32];
  const int tid = threadIdx.x;
  const int ps = 1 << a.ps_log2;
  int len = 0, add = 0, have = 0, need = 0;
  bool good = true;
  const int used0 = __ldcg(a.used);
  if (tid < a.members) {
    len = __ldcg(a.lens + tid);
    add = __ldg(a.add + tid);
    const long long room = (long long)a.max_blocks << a.ps_log2;
    // a member out of use (negative length) may not grow
    good = add >= 0 && (len >= 0 || add == 0) && (long long)(len < 0 ? 0 : len) + add <= room &&
           (!kRows || add <= a.rows);
    if (good && len >= 0) {
      have = (int)(((long long)len + ps - 1) >> a.ps_log2);
      need = (int)(((long long)len + add + ps - 1) >> a.ps_log2);
    } else if (!good) {
      add = 0;
    }
  }
  long long tok = add;
  int pages = need - have;
  block_scan(&tok, &pages, wt, wp);
  p.tok_end[tid] = tok;
  p.page_end[tid] = pages;
  p.len[tid] = len;
  p.have[tid] = have;
  const bool all_good = __syncthreads_and(good);
  const long long total = p.tok_end[kThreads - 1];
  const int new_pages = p.page_end[kThreads - 1];
  const bool ok = all_good && total <= a.capacity && used0 >= 0 &&
                  (long long)used0 + new_pages <= a.num_free;
  if (tid == 0) {
    p.used0 = used0;
    if (!ok && commit) ls_report(a.err, LS_DEVERR_CHECK);
  }
  __syncthreads();
  if (fill) {
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + tid) * kPerThread; i < a.capacity;
         i += (int64_t)gridDim.x * kChunk) {
      int32_t slot[kPerThread], pos[kPerThread];
      int m = -1;
      long long begin = 0, end = 0;
      // packed, the tokens end at `total`; with rows every one belongs to a member
      const long long stop = kRows ? a.capacity : total;
#pragma unroll
      for (int e = 0; e < kPerThread; ++e) {
        slot[e] = -1;
        pos[e] = 0;
        const long long t = i + e;
        if (!ok || t >= stop) continue;
        if (kRows) {
          m = (int)(t / a.rows);
          end = (long long)(m + 1) * a.rows;
          begin = end - (p.tok_end[m] - (m ? p.tok_end[m - 1] : 0));
          if (t < begin) continue;
        } else if (m < 0) {  // first member whose tokens end behind t
          int lo = 0, hi = a.members - 1;
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (p.tok_end[mid] > t) hi = mid; else lo = mid + 1;
          }
          m = lo;
          begin = m ? p.tok_end[m - 1] : 0;
          end = p.tok_end[m];
        }
        while (t >= end) {
          ++m;
          begin = end;
          end = p.tok_end[m];
        }
        const int at = p.len[m] + (int)(t - begin);
        const int32_t page = page_of(a, p, m, at >> a.ps_log2);
        pos[e] = a.pos0 + at;
        if ((uint32_t)page < (uint32_t)a.num_pages)
          slot[e] = (page << a.ps_log2) + (at & (ps - 1));
        else
          ls_report(a.err, LS_DEVERR_CHECK);
      }
      if (i + kPerThread <= a.capacity) {
        *reinterpret_cast<int4*>(a.slots + i) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      } else {
        for (int e = 0; i + e < a.capacity; ++e) a.slots[i + e] = slot[e];
      }
      if (a.pos) {
        const bool vec = i + kPerThread <= a.capacity && (a.capacity & 3) == 0;
        for (int x = 0; x < a.axes; ++x) {
          int32_t* row = a.pos + x * a.capacity + i;
          if (vec) {
            *reinterpret_cast<int4*>(row) = make_int4(pos[0], pos[1], pos[2], pos[3]);
          } else {
            for (int e = 0; e < kPerThread && i + e < a.capacity; ++e) row[e] = pos[e];
          }
        }
      }
    }
    if (ok) {
      for (int i = blockIdx.x * kThreads + tid; i < new_pages; i += gridDim.x * kThreads) {
        int lo = 0, hi = a.members - 1;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (p.page_end[mid] > i) hi = mid; else lo = mid + 1;
        }
        const int before = lo ? p.page_end[lo - 1] : 0;
        a.table[(int64_t)lo * a.max_blocks + p.have[lo] + i - before] =
            __ldg(a.free_list + used0 + i);
      }
    }
  }
  if (commit && blockIdx.x == 0) {
    if (tid < a.members) a.lens_out[tid] = ok ? len + add : len;
    if (tid == 0) *a.used_out = ok ? used0 + new_pages : used0;
  }
}

}  // namespace

cudaError_t ls_launch_extend_pages(const LsExtendArgs& a, int sms, cudaStream_t st) {
  int64_t blocks = (a.capacity + kChunk - 1) / kChunk;
  if (blocks < 1) blocks = 1;
  if (blocks > sms) blocks = sms;
  auto meets = [](const int32_t* p, int64_t n, const int32_t* q, int64_t m) { return p < q + m && q < p + n; };
  bool in_place = false;
  const struct { const int32_t* p; int64_t n; } in[] = {{a.lens, a.members}, {a.add, a.members}, {a.used, 1}};
  for (const auto& i : in)
    in_place = in_place || meets(a.lens_out, a.members, i.p, i.n) || meets(a.used_out, 1, i.p, i.n);
  const bool one = blocks == 1 || !in_place;
  const auto kernel = a.rows ? extend_pages_kernel<true> : extend_pages_kernel<false>;
  kernel<<<(unsigned)blocks, kThreads, 0, st>>>(a, 1, one ? 1 : 0);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ls_note_launch();
  if (!one) {
    kernel<<<1, kThreads, 0, st>>>(a, 0, 1);
    e = cudaGetLastError();
    if (e == cudaSuccess) ls_note_launch();
  }
  return e;
}
