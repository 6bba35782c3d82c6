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
// extend_pages is bound by a launch and one dependent chain (lengths, two scans, a search, a page, a
// slot): one token for each of 8 members 4.0 us, 282,000 tokens for 64 members 5.2 us, of
// which the 2.2 MB of slots and positions are 0.3 us at the copy's rate.
//
// Below: pages given back at the end of sequences, and shared by branches of a sequence.
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
    add = !kRows || a.add ? __ldg(a.add + tid) : len < 0 ? 0 : a.rows;
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
    if (tid < a.members) {
      a.lens_out[tid] = ok ? len + add : len;
      if (kRows && a.added) a.added[tid] = ok ? add : 0;
    }
    if (tid == 0) *a.used_out = ok ? used0 + new_pages : used0;
  }
}

// ---------------------------------------------------------------- pages given back
//
// Member m keeps its first new_len tokens; the pages behind them lose it as an owner.  A page
// that no owner is left of goes back to the free list, which is a stack: the freed pages, in
// member and block order, become its entries [used - freed, used).
//
// shared[page] counts a page's owners besides the first, so a page that extend_pages has just
// taken is at its right count, 0.  A call may drop several owners of a page at once; which of
// its entries stands for the page in the free list must not depend on who came first.  So the
// drops are counted into shared (integer atomics: the sum is the same in any order), a page
// that lost all its owners ends at -1, and among its entries the first one is found by a
// maximum over INT_MIN + (entries - place), kept in shared as well until the end.
//
// One block: the counts of all entries have to meet before the first is written.  A decode
// step's drafts free about a page a member; 8,192 entries take eight rounds of each phase.

struct Drops {
  int end[kThreads];   // entries up to and including the member
  int need[kThreads];  // its first dropped block
};

__global__ void __launch_bounds__(kThreads) trim_pages_kernel(const LsShareArgs a,
                                                              const int32_t* __restrict__ new_lens) {
  __shared__ Drops d;
  __shared__ long long wt[32];
  __shared__ int wp[32];
  __shared__ int batch[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ps = 1 << a.ps_log2, used0 = *a.used;
  int len = -1, keep = -1, have = 0, need = 0;
  bool good = true;
  if (tid < a.members) {
    len = a.lens[tid];
    keep = new_lens[tid];
    good = len < 0 ? keep < 0 : keep <= len && len <= ((long long)a.max_blocks << a.ps_log2);
    if (good) {
      have = len > 0 ? (int)(((long long)len + ps - 1) >> a.ps_log2) : 0;
      need = keep > 0 ? (int)(((long long)keep + ps - 1) >> a.ps_log2) : 0;
    }
  }
  long long tok = 0;
  int drops = have - need;
  block_scan(&tok, &drops, wt, wp);
  d.end[tid] = drops;
  d.need[tid] = need;
  good = __syncthreads_and(good) && used0 >= 0 && used0 <= a.num_free;
  const int total = d.end[kThreads - 1];
  auto page_at = [&](int j) {  // the page of entry j
    int lo = 0, hi = a.members - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (d.end[mid] > j) hi = mid; else lo = mid + 1;
    }
    return a.table[(int64_t)lo * a.max_blocks + d.need[lo] + j - (lo ? d.end[lo - 1] : 0)];
  };
  auto in_pool = [&](int page) { return (uint32_t)page < (uint32_t)a.num_pages; };
  int freed = total;
  if (good) {
    bool fine = true;
    for (int j = tid; j < total; j += kThreads) {
      const int page = page_at(j);
      if (!in_pool(page)) fine = false;
      else if (a.shared) atomicSub(a.shared + page, 1);
    }
    good = __syncthreads_and(fine);
    bool undo = !good;
    if (a.shared && good) {
      fine = true;
      int n = 0;
      for (int j = tid; j < total; j += kThreads)
        if (__ldcg(a.shared + page_at(j)) < -1) fine = false;  // more owners dropped than it had
      // a member cut inside a page that others still read would write there next
      if (keep > 0 && keep < len && (keep & (ps - 1))) {
        const int page = a.table[(int64_t)tid * a.max_blocks + (keep >> a.ps_log2)];
        if (in_pool(page) && __ldcg(a.shared + page) > 0) fine = false;
      }
      good = __syncthreads_and(fine);
      undo = !good;
      if (good) {
        for (int j = tid; j < total; j += kThreads) {
          int32_t* c = a.shared + page_at(j);
          if (__ldcg(c) < 0) __stcg(c, INT32_MIN);  // every entry of the page writes the same
        }
        __syncthreads();
        for (int j = tid; j < total; j += kThreads) {
          int32_t* c = a.shared + page_at(j);
          if (__ldcg(c) < 0) atomicMax(c, INT32_MIN + (total - j));
        }
        __syncthreads();
        for (int j = tid; j < total; j += kThreads)
          n += __ldcg(a.shared + page_at(j)) == INT32_MIN + (total - j);
        int sum = n;
        tok = 0;
        __syncthreads();
        block_scan(&tok, &sum, wt, wp);
        freed = wp[31];
        if (freed > used0) {  // pages that were never taken: the counts before the drops again
          good = false;
          undo = true;
          for (int j = tid; j < total; j += kThreads) {
            int32_t* c = a.shared + page_at(j);
            if (__ldcg(c) < 0) __stcg(c, -1);
          }
          __syncthreads();
        }
      }
    } else if (good && freed > used0) {
      good = false;
    }
    if (undo && a.shared)
      for (int j = tid; j < total; j += kThreads) {
        const int page = page_at(j);
        if (in_pool(page)) atomicAdd(a.shared + page, 1);
      }
  }
  if (good) {
    int before = used0 - freed;
    for (int j0 = 0; j0 < total; j0 += kThreads) {
      const int j = j0 + tid, page = j < total ? page_at(j) : -1;
      const bool mine = j < total && (!a.shared || __ldcg(a.shared + page) == INT32_MIN + (total - j));
      const uint32_t mask = __ballot_sync(0xffffffffu, mine);
      if (lane == 0) batch[warp] = __popc(mask);
      __syncthreads();
      int at = before;
#pragma unroll
      for (int w = 0; w < 32; ++w) {
        if (w < warp) at += batch[w];
        before += batch[w];
      }
      if (mine) a.free_list[at + __popc(mask & ((1u << lane) - 1))] = page;
      __syncthreads();
    }
    if (a.shared) {
      for (int j = tid; j < total; j += kThreads) {
        int32_t* c = a.shared + page_at(j);
        if (__ldcg(c) < 0) __stcg(c, 0);
      }
    }
  }
  if (tid < a.members) a.lens_out[tid] = !good || len < 0 ? len : max(keep, -1);
  if (tid == 0) {
    *a.used_out = good ? used0 - freed : used0;
    if (!good) ls_report(a.err, LS_DEVERR_CHECK);
  }
}

// ---------------------------------------------------------------- pages shared
//
// Member m, out of use or empty, becomes a branch of member src[m]'s first keep[m] tokens: the
// whole pages are shared, the rows of a partial last one are to be copied to a page of its own
// (from the free list, in member order), which `copies` says to copy_pages.  One block, as for
// trim_pages; the entries of a branch's table are written and counted by all of its threads.
__global__ void __launch_bounds__(kThreads) fork_pages_kernel(const LsShareArgs a,
                                                              const int32_t* __restrict__ src,
                                                              const int32_t* __restrict__ keep,
                                                              int32_t* copies) {
  __shared__ int end[kThreads], from_member[kThreads];
  __shared__ long long wt[32];
  __shared__ int wp[32];
  const int tid = threadIdx.x;
  const int used0 = *a.used;
  int len = -1, of = -1, n = 0, whole = 0, part = 0, source = -1;
  bool good = true;
  if (tid < a.members) {
    len = a.lens[tid];
    of = src[tid];
    if (of >= 0) {
      good = of < a.members && of != tid && len <= 0;
      if (good) {
        const int olen = a.lens[of];
        n = keep ? keep[tid] : olen;
        good = olen >= 0 && src[of] < 0 && n >= 0 && n <= olen &&
               olen <= ((long long)a.max_blocks << a.ps_log2);
      }
      if (good) {
        whole = n >> a.ps_log2;
        part = n & ((1 << a.ps_log2) - 1);
        if (part) {
          source = a.table[(int64_t)of * a.max_blocks + whole];
          good = (uint32_t)source < (uint32_t)a.num_pages;
        }
      } else {
        n = 0;
      }
    }
  }
  const bool fresh = good && part > 0;
  long long entries = good ? whole : 0;
  int taken = fresh;
  block_scan(&entries, &taken, wt, wp);
  end[tid] = (int)entries;
  from_member[tid] = of;
  good = __syncthreads_and(good) && used0 >= 0 && wp[31] <= a.num_free - used0;
  const int total = end[kThreads - 1], pages = wp[31];
  auto entry = [&](int j, int* member) {  // block of the branch that entry j is
    int lo = 0, hi = a.members - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (end[mid] > j) hi = mid; else lo = mid + 1;
    }
    *member = lo;
    return j - (lo ? end[lo - 1] : 0);
  };
  int page = -1;
  bool fine = true;
  if (good) {
    if (fresh) {
      page = a.free_list[used0 + taken - 1];
      fine = (uint32_t)page < (uint32_t)a.num_pages;
    }
    for (int j = tid; j < total; j += kThreads) {
      int m;
      const int b = entry(j, &m);
      const int32_t x = a.table[(int64_t)from_member[m] * a.max_blocks + b];
      if ((uint32_t)x >= (uint32_t)a.num_pages) fine = false;
    }
  }
  good = __syncthreads_and(fine) && good;
  if (good) {
    for (int j = tid; j < total; j += kThreads) {
      int m;
      const int b = entry(j, &m);
      const int32_t x = a.table[(int64_t)from_member[m] * a.max_blocks + b];
      a.table[(int64_t)m * a.max_blocks + b] = x;
      atomicAdd(a.shared + x, 1);
    }
    if (fresh) a.table[(int64_t)tid * a.max_blocks + whole] = page;
  }
  if (tid < a.members) {
    const bool copy = good && fresh;
    copies[tid] = copy ? source : -1;
    copies[a.members + tid] = copy ? page : -1;
    copies[2 * a.members + tid] = copy ? part : 0;
    a.lens_out[tid] = good && of >= 0 ? n : len;
  }
  if (tid == 0) {
    *a.used_out = good ? used0 + pages : used0;
    if (!good) ls_report(a.err, LS_DEVERR_CHECK);
  }
}

}  // namespace

cudaError_t ls_launch_trim_pages(const LsShareArgs& a, const int32_t* new_lens, cudaStream_t st) {
  trim_pages_kernel<<<1, kThreads, 0, st>>>(a, new_lens);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ls_note_launch();
  return e;
}

cudaError_t ls_launch_fork_pages(const LsShareArgs& a, const int32_t* src, const int32_t* keep,
                                 int32_t* copies, cudaStream_t st) {
  fork_pages_kernel<<<1, kThreads, 0, st>>>(a, src, keep, copies);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ls_note_launch();
  return e;
}

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
