// Page tables of the cache: rows of pages with a count of the table entries that name each page.
//
// A page whose count is 0 is free, so the counts are all the state there is, and pages are given out lowest first.
// Everything here is a few thousand integers; the calls are bound by launches and dependent reads, but for the copies
// of rows (growth) and pages (compaction), which HBM bounds: 4096 pages of 256 KB, 0.6 in use, take 79 us for 515 MB
// (6.5 TB/s), 89 with the plan.  Each by itself, a fork of a prompt of 32K tokens to 19 rows and a trim of 64 rows take 2 us,
// the growth of 32 rows by a token 6.2.
#include <stdint.h>

#include <atomic>

#include "bsa_pages.h"
#include "bsa_tree.cuh"

namespace bsa {
namespace {

constexpr int kThreads = 256;
constexpr int kPlanThreads = 1024;
constexpr int kSms = 152;
constexpr int kMarks = 1 << 18;  // most bits by which growth knows last pages of two sequences (32 KB)
constexpr int kWide = 1 << 18;   // pages of one sequence from which on a sum of 4096 of them is taken in 64 bits
constexpr int kHeld = 4;  // neighbouring pages of a planning thread, of which the first round's counts stay in registers

// Threads of a planning CTA: a round takes all pages, and all sequences, up to kPlanThreads (fewer threads meet sooner).
int plan_threads(int pages, int batch) {
  const int want = (pages + kHeld - 1) / kHeld > batch ? (pages + kHeld - 1) / kHeld : batch;
  return want >= kPlanThreads ? kPlanThreads : want <= 128 ? 128 : (want + 31) / 32 * 32;
}

__device__ __forceinline__ void report(int32_t *status, bsa_status what) {
  if (status != nullptr) atomicCAS(status, 0, static_cast<int32_t>(what));
}

// The cached tokens of row b, 0 (and a report) where its row of the table cannot hold them.
__device__ __forceinline__ int held(const int32_t *cached, int b, int page_shift, int stride, int32_t *status) {
  const int n = cached[b];
  if (n >= 0 && (n == 0 || (n - 1) >> page_shift < stride)) return n;
  report(status, BSA_ERR_INVALID_ARG);
  return 0;
}
__device__ __forceinline__ int pages_of(int tokens, int page_shift) {
  return tokens == 0 ? 0 : ((tokens - 1) >> page_shift) + 1;
}
// `by` table entries more (or one less) name `page`, which one does: a count below 1 is not right, and stays as it is.
// (Right counts are above 0 whenever this looks, as the entry looked at is among those counted.)
__device__ __forceinline__ void count_page(int32_t *refs, int pages, int page, int by, int32_t *status) {
  if (page < 0 || page >= pages) {
    report(status, BSA_ERR_INVALID_ARG);
  } else if (atomicAdd(refs + page, by) < 1) {
    atomicSub(refs + page, by);
    report(status, BSA_ERR_INVALID_ARG);
  }
}

// ---------------------------------------------------------------- fork, trim

// blockIdx.y < batch: a row of the old table, whose pages are named once less, and once more for every new row made
// of it (one atomic for the difference); the rest: a row of the new table.
__global__ void __launch_bounds__(kThreads) fork_kernel(const ForkArgs a) {
  const int b = blockIdx.y;
  if (b < a.batch) {
    int uses = 0;
    for (int base = 0; base < a.batch_out; base += kThreads) {
      const int j = base + static_cast<int>(threadIdx.x);
      uses += __syncthreads_count(j < a.batch_out && a.source[j] == b);
    }
    const int have = pages_of(held(a.cached, b, a.page_shift, a.stride, a.status), a.page_shift);
    if (uses == 1) return;
    for (int j = blockIdx.x * kThreads + threadIdx.x; j < have; j += gridDim.x * kThreads)
      count_page(a.refs, a.pages, a.table[static_cast<size_t>(b) * a.stride + j], uses - 1, a.status);
    return;
  }
  const int row = b - a.batch;
  int from = a.source[row];
  if (from < -1 || from >= a.batch) {
    report(a.status, BSA_ERR_INVALID_ARG);
    from = -1;
  }
  const int n = from < 0 ? 0 : held(a.cached, from, a.page_shift, a.stride, a.status);
  const int have = pages_of(n, a.page_shift);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.cached_out[row] = n;
  for (int j = blockIdx.x * kThreads + threadIdx.x; j < a.stride; j += gridDim.x * kThreads)
    a.table_out[static_cast<size_t>(row) * a.stride + j] = j < have ? a.table[static_cast<size_t>(from) * a.stride + j] : -1;
}

__global__ void __launch_bounds__(kThreads) trim_kernel(const TrimArgs a) {
  const int b = blockIdx.x;
  const int n = held(a.cached, b, a.page_shift, a.stride, a.status), keep = a.keep[b];
  const bool bad = keep < 0 || keep > n || a.cached[b] != n;  // (a length that its row cannot hold reads as 0)
  __syncthreads();  // everyone has read the length
  if (bad) {
    if (threadIdx.x == 0) report(a.status, BSA_ERR_INVALID_ARG);
    return;
  }
  const int have = pages_of(n, a.page_shift);
  for (int j = pages_of(keep, a.page_shift) + threadIdx.x; j < have; j += kThreads) {
    int32_t *entry = a.table + static_cast<size_t>(b) * a.stride + j;
    count_page(a.refs, a.pages, *entry, -1, a.status);
    *entry = -1;
  }
  if (threadIdx.x == 0) a.cached[b] = keep;
}

// ---------------------------------------------------------------- sums over a planning block

// The sum of the values of the threads before this one; *total the whole sum.  `warps`: [33] of shared memory.
__device__ __forceinline__ int scan_block(int value, int *warps, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = value;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();  // the last sums have been read
  if (lane == 31) warps[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < blockDim.x >> 5 ? warps[lane] : 0;
    int run = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += up;
    }
    warps[lane] = run - w;
    if (lane == 31) warps[32] = run;
  }
  __syncthreads();
  *total = warps[32];
  return warps[warp] + inc - value;
}

// ---------------------------------------------------------------- growth

// The counts of this thread's pages of a round, INT_MIN behind the pool's end.
struct Held {
  int refs[kHeld];
};
__device__ __forceinline__ Held held_pages(const int32_t *refs, int pages, int round) {
  Held h;
#pragma unroll
  for (int e = 0; e < kHeld; ++e) {
    const int p = (round * static_cast<int>(blockDim.x) + static_cast<int>(threadIdx.x)) * kHeld + e;
    h.refs[e] = p < pages ? refs[p] : INT32_MIN;
  }
  return h;
}
// Bits for a pool's pages: as many, or kMarks, of which page p takes bit p % kMarks.
__host__ __device__ __forceinline__ int mark_words(int pages) { return ((pages < kMarks ? pages : kMarks) + 31) / 32; }
__device__ __forceinline__ int rounds_of(int pages) { return (pages + blockDim.x * kHeld - 1) / (blockDim.x * kHeld); }

// One CTA plans: who needs how many pages (a copy of a shared last page among them, unless this is the last sequence
// that holds it), whether there are enough, and which; sequences and pages in ascending order, so that the outcome is
// that of one sequence after the other.
__global__ void __launch_bounds__(kPlanThreads) grow_plan_kernel(const GrowArgs a) {
  extern __shared__ int sm[];
  // [batch] the partial last page that gets tokens or -1; [batch] where the first new page goes, times 2, and whether
  // that is a copy; [batch + 1] the first new page; a bit per page that is somebody's last and counts once
  int *last = sm, *goes = sm + a.batch, *first = goes + a.batch, *marks = first + a.batch + 1;
  __shared__ int warps[33];
  __shared__ int carry;
  __shared__ unsigned long long wide;  // pages of the sequences that need kWide or more
  const int tid = threadIdx.x, threads = blockDim.x, shift = a.c.page_shift, mask = a.c.page - 1;
  launch_next();
  struct Seq {
    int n, g, page, refs;  // tokens, those it grows by, its partial last page (-1: none) and the count of that
  };
  auto read = [&](int b) -> Seq {
    Seq s{held(a.cached, b, shift, a.stride, a.status), 0, -1, 0};
    if (a.cached[b] != s.n) return s;  // (reported)
    const int t0 = a.cu[b], t1 = a.cu[b + 1];
    if (t0 < 0 || t1 < t0 || t1 > a.total) {
      report(a.status, BSA_ERR_INVALID_ARG);
      return s;
    }
    s.g = a.grow == nullptr ? t1 - t0 : a.grow[b];
    if (s.g < 0 || s.g > t1 - t0 || s.n > INT32_MAX - s.g || pages_of(s.n + s.g, shift) > a.stride) {
      report(a.status, BSA_ERR_INVALID_ARG);
      s.g = 0;
    }
    if (s.g > 0 && (s.n & mask) != 0) {
      s.page = a.table[static_cast<size_t>(b) * a.stride + (s.n >> shift)];
      if (s.page >= 0 && s.page < a.c.pages) s.refs = a.refs[s.page];
      if (s.refs < 1) {  // none, or one that is free for others to get
        report(a.status, BSA_ERR_INVALID_ARG);
        s.page = -1;
        s.g = 0;
      }
    }
    return s;
  };
  const Held round0 = held_pages(a.refs, a.c.pages, 0);
  for (int i = tid; i < mark_words(a.c.pages); i += threads) marks[i] = 0;
  Seq seq0{0, 0, -1, 0};  // the first round's stays in registers
  if (tid < a.batch) seq0 = read(tid);
  __syncthreads();
  bool met = false;       // a page that counts once was marked before: two sequences name it (or pages kMarks apart)
  for (int b = tid; b < a.batch; b += threads) {
    const Seq s = b == tid ? seq0 : read(b);
    last[b] = s.page;
    if (s.refs == 1) {
      const int bit = s.page & (kMarks - 1);
      met |= (atomicOr(marks + (bit >> 5), 1 << (bit & 31)) >> (bit & 31) & 1) != 0;
    }
  }
  if (tid == 0) carry = 0, wide = 0;
  met = __syncthreads_or(met) != 0;
  for (int base = 0; base < a.batch; base += threads) {
    const int b = base + tid;
    int need = 0;
    if (b < a.batch) {
      Seq s = base == 0 ? seq0 : read(b);
      int earlier = 0;
      if (s.refs > 1 || (s.refs == 1 && met))
        for (int x = 0; x < b; ++x) earlier += last[x] == s.page ? 1 : 0;
      if (s.page >= 0 && s.refs - earlier < 1) {  // more sequences hold it than are counted: the first of them grow
        report(a.status, BSA_ERR_INVALID_ARG);
        s.g = 0;
        if (base == 0) seq0.g = 0;
      }
      const bool copy = s.refs - earlier > 1;
      need = s.g == 0 ? 0 : pages_of(s.n + s.g, shift) - pages_of(s.n, shift) + (copy ? 1 : 0);
      if (need >= kWide) atomicAdd(&wide, static_cast<unsigned long long>(need));
      goes[b] = 2 * (pages_of(s.n, shift) - (copy ? 1 : 0)) + (copy ? 1 : 0);
      a.jobs[b] = GrowJob{s.g > 0 ? s.n : -1, copy ? s.page : -1, -1, copy ? s.n & mask : 0};
    }
    int total;
    const int before = scan_block(need, warps, &total);
    if (b < a.batch) first[b] = carry + before;
    __syncthreads();
    if (tid == 0) carry += total;
    __syncthreads();
  }
  const int total = carry;
  if (tid == 0) first[a.batch] = total;
  __syncthreads();

  // the free pages, lowest first
  auto free_of = [&](const Held &h) {
    int n = 0;
#pragma unroll
    for (int e = 0; e < kHeld; ++e) n += h.refs[e] == 0 ? 1 : 0;
    return n;
  };
  auto give = [&](const Held &h, int round, int k) {  // k: the free pages before this thread's
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      if (h.refs[e] != 0) continue;
      const int p = (round * threads + tid) * kHeld + e;
      if (k < total) {
        int lo = 0, hi = a.batch - 1;
        while (lo < hi) {  // the last sequence whose first new page is at or before k: the one that gets it
          const int mid = (lo + hi + 1) >> 1;
          if (first[mid] <= k) lo = mid;
          else hi = mid - 1;
        }
        const int to = goes[lo];
        if ((to & 1) != 0 && k == first[lo]) a.jobs[lo].to = p;
        a.table[static_cast<size_t>(lo) * a.stride + (to >> 1) + k - first[lo]] = p;
        a.refs[p] = 1;
      }
      ++k;
    }
  };
  auto nobody = [&]() {  // not enough pages: nobody grows
    if (tid == 0) report(a.status, BSA_ERR_WORKSPACE);
    for (int b = tid; b < a.batch; b += threads) a.jobs[b] = GrowJob{-1, -1, -1, 0};
  };
  // offsets that descend name a token in several sequences, whose pages may add up to more than 32 bits hold
  if (wide > static_cast<unsigned long long>(a.c.pages)) return nobody();
  if (total > 0) {
    int n;
    const int k0 = scan_block(free_of(round0), warps, &n);
    const int rounds = rounds_of(a.c.pages);
    int found = n;
    for (int r = 1; r < rounds && found < total; ++r) {
      int more;
      scan_block(free_of(held_pages(a.refs, a.c.pages, r)), warps, &more);
      found += more;
    }
    if (found < total) return nobody();
    give(round0, 0, k0);
    for (int r = 1; n < total; ++r) {
      const Held h = held_pages(a.refs, a.c.pages, r);
      int more;
      const int k = n + scan_block(free_of(h), warps, &more);
      give(h, r, k);
      n += more;
    }
  }
  for (int base = 0; base < a.batch; base += threads) {
    const int b = base + tid;
    if (b >= a.batch) break;
    const int from = (goes[b] & 1) != 0 ? last[b] : -1;
    if (from >= 0) atomicSub(a.refs + from, 1);
    const int n = base == 0 ? seq0.n : held(a.cached, b, shift, a.stride, nullptr);
    const int g = base == 0 ? seq0.g : a.jobs[b].start < 0 ? 0 : a.grow == nullptr ? a.cu[b + 1] - a.cu[b] : a.grow[b];
    if (g > 0) a.cached[b] = n + g;
  }
}

// 16 bytes at a time, or bytes where the ends are not on such boundaries.
__device__ __forceinline__ void copy_bytes(uint8_t *to, const uint8_t *from, int bytes) {
  const int wide = ((reinterpret_cast<uintptr_t>(to) | reinterpret_cast<uintptr_t>(from)) & 15) == 0 ? bytes / 16 : 0;
  for (int i = threadIdx.x; i < wide; i += blockDim.x)
    reinterpret_cast<uint4 *>(to)[i] = __ldg(reinterpret_cast<const uint4 *>(from) + i);
  for (int i = wide * 16 + threadIdx.x; i < bytes; i += blockDim.x) to[i] = __ldg(from + i);
}

// The first blocks write the slots of the new tokens; then one for every (sequence, KV head, K or V) copies the rows
// of a shared last page.
__global__ void __launch_bounds__(kThreads) grow_rows_kernel(const GrowArgs a, int slot_blocks) {
  after_previous_kernel();
  if (static_cast<int>(blockIdx.x) < slot_blocks) {
    for (int t = blockIdx.x * kThreads + threadIdx.x; t < a.total; t += slot_blocks * kThreads) {
      int lo = 0, hi = a.batch - 1;
      while (lo < hi) {  // the last sequence that begins at or before t
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(a.cu + mid) <= t) lo = mid;
        else hi = mid - 1;
      }
      const int t0 = __ldg(a.cu + lo), t1 = __ldg(a.cu + lo + 1);
      if (t < t0 || t >= t1) continue;  // past the last sequence: left as it was
      const GrowJob job = a.jobs[lo];
      int slot = -1;
      if (job.start >= 0) {
        const int g = a.cached[lo] - job.start, rank = a.rank == nullptr ? t - t0 : __ldg(a.rank + t);
        if (rank >= 0 && rank < g) {
          const int pos = job.start + rank;
          const int page = a.table[static_cast<size_t>(lo) * a.stride + (pos >> a.c.page_shift)];
          slot = (page << a.c.page_shift) + (pos & (a.c.page - 1));
        }
      }
      a.slots[t] = slot;
    }
    return;
  }
  const int x = blockIdx.x - slot_blocks, per = 2 * a.c.hkv;
  const int b = x / per, head = x % per / 2, kv = x & 1;
  const GrowJob job = a.jobs[b];
  if (job.to < 0) return;
  const size_t tile_from = static_cast<size_t>(job.from) * a.c.hkv + head;
  const size_t tile_to = static_cast<size_t>(job.to) * a.c.hkv + head;
  const size_t codes = static_cast<size_t>(a.c.page) * a.c.row;
  copy_bytes(a.planes[kv] + tile_to * codes, a.planes[kv] + tile_from * codes, job.rows * a.c.row);
  if (a.c.per_row == 0) return;
  const size_t scales = static_cast<size_t>(a.c.page) * a.c.per_row;
  uint8_t *to = a.planes[2 + kv] + tile_to * scales;
  const uint8_t *from = a.planes[2 + kv] + tile_from * scales;
  copy_bytes(to, from, job.rows);
  if (a.c.per_row > 1) copy_bytes(to + a.c.page, from + a.c.page, job.rows * (a.c.per_row - 1));
}

// ---------------------------------------------------------------- compaction

// One CTA: with L pages in use, the pages in use from L on go, in order, to the free ones below L.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const CompactArgs a) {
  __shared__ int warps[33];
  const int tid = threadIdx.x, threads = blockDim.x, pages = a.c.pages, rounds = rounds_of(pages);
  int *holes = a.work + 4, *moved = holes + pages, *to = moved + pages;
  launch_next();
  const Held round0 = held_pages(a.refs, pages, 0);
  int live = 0;
  for (int r = 0; r < rounds; ++r) {
    const Held h = r == 0 ? round0 : held_pages(a.refs, pages, r);
    int used = 0, n;
#pragma unroll
    for (int e = 0; e < kHeld; ++e) used += h.refs[e] > 0 ? 1 : 0;
    scan_block(used, warps, &n);
    live += n;
  }
  int nh = 0, nm = 0;
  for (int r = 0; r < rounds; ++r) {
    const Held h = r == 0 ? round0 : held_pages(a.refs, pages, r);
    const int p0 = (r * threads + tid) * kHeld;
    int mine = 0, n;  // holes, and times 2^16 pages that move (at most 4096 of each a round)
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      const int p = p0 + e;
      mine += p < live && h.refs[e] <= 0 ? 1 : p >= live && h.refs[e] > 0 ? 0x10000 : 0;
    }
    const int k = scan_block(mine, warps, &n);
    int hole = nh + (k & 0xFFFF), move = nm + (k >> 16);
#pragma unroll
    for (int e = 0; e < kHeld; ++e) {
      const int p = p0 + e;
      if (p >= pages) break;
      if (p < live && h.refs[e] <= 0) holes[hole++] = p;
      if (p >= live && h.refs[e] > 0) moved[move++] = p;
      if (h.refs[e] <= 0) to[p] = -1;  // (no entry should name it: below L it gets another's page)
      else if (p < live) to[p] = p;
    }
    nh += n & 0xFFFF;
    nm += n >> 16;
  }
  __syncthreads();
  for (int i = tid; i < nm; i += threads) {
    const int src = moved[i], dst = holes[i];
    to[src] = dst;
    a.refs[dst] = a.refs[src];
    a.refs[src] = 0;
  }
  if (tid == 0) {
    a.work[0] = nm;
    *a.live = live;
  }
}

// The first blocks rewrite the tables, all copy pages.
__global__ void __launch_bounds__(kThreads) compact_move_kernel(const CompactArgs a) {
  after_previous_kernel();
  const int pages = a.c.pages;
  const int *holes = a.work + 4, *moved = holes + pages, *to = moved + pages;
  const long long entries = static_cast<long long>(a.batch) * a.stride;
  for (long long e = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; e < entries;
       e += static_cast<long long>(gridDim.x) * kThreads) {
    const int b = static_cast<int>(e / a.stride), j = static_cast<int>(e % a.stride);
    if (j >= pages_of(held(a.cached, b, a.c.page_shift, a.stride, a.status), a.c.page_shift)) continue;
    const int p = a.table[e];
    const int q = p >= 0 && p < pages ? to[p] : -1;
    if (q < 0) report(a.status, BSA_ERR_INVALID_ARG);
    else if (q != p) a.table[e] = q;
  }
  const int moves = a.work[0];
  // a block takes pieces of a page's part of an array, codes first; four loads of a thread under way
  constexpr int kPiece = 4 * kThreads;  // times 16 bytes
  const int n16[2] = {static_cast<int>(static_cast<size_t>(a.c.hkv) * a.c.page * a.c.row / 16),
                      static_cast<int>(static_cast<size_t>(a.c.hkv) * a.c.page * a.c.per_row / 16)};
  const int codes = (n16[0] + kPiece - 1) / kPiece, scales = (n16[1] + kPiece - 1) / kPiece, pieces = 2 * (codes + scales);
  for (long long e = blockIdx.x; e < static_cast<long long>(moves) * pieces; e += gridDim.x) {
    const int i = static_cast<int>(e / pieces);
    int x = static_cast<int>(e - static_cast<long long>(i) * pieces);
    const int kind = x < 2 * codes ? 0 : 1, each = kind == 0 ? codes : scales, n = n16[kind];
    x -= kind == 0 ? 0 : 2 * codes;
    const int kv = x >= each ? 1 : 0;
    uint4 *plane = reinterpret_cast<uint4 *>(a.planes[2 * kind + kv]);
    const uint4 *from = plane + static_cast<size_t>(moved[i]) * n;
    uint4 *to_page = plane + static_cast<size_t>(holes[i]) * n;
    const int at = (x - kv * each) * kPiece + threadIdx.x;
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (at + u * kThreads < n) v[u] = __ldcs(from + at + u * kThreads);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (at + u * kThreads < n) __stcs(to_page + at + u * kThreads, v[u]);
  }
}

}  // namespace

cudaError_t launch_fork(const ForkArgs &a, cudaStream_t stream) {
  const int x = (a.stride + kThreads - 1) / kThreads;
  fork_kernel<<<dim3(x < 8 ? x : 8, a.batch + a.batch_out), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_trim(const TrimArgs &a, cudaStream_t stream) {
  trim_kernel<<<a.batch, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

size_t grow_workspace_bytes(int batch) { return static_cast<size_t>(batch) * sizeof(GrowJob); }

cudaError_t launch_grow(const GrowArgs &a, cudaStream_t stream) {
  auto smem_of = [](int batch, int pages) { return (3 * static_cast<size_t>(batch) + 1 + mark_words(pages)) * sizeof(int); };
  static std::atomic<uint64_t> done{0};
  cudaError_t e = set_up(grow_plan_kernel, smem_of(kMaxDecodeRows, kMarks), 0, done);
  if (e != cudaSuccess) return e;
  grow_plan_kernel<<<1, plan_threads(a.c.pages, a.batch), smem_of(a.batch, a.c.pages), stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int want = (a.total + kThreads - 1) / kThreads, slot_blocks = want < kSms ? want : kSms;
  return launch_after(grow_rows_kernel, dim3(slot_blocks + a.batch * a.c.hkv * 2), kThreads, 0, stream, a, slot_blocks);
}

size_t compact_workspace_bytes(int pages) { return (4 + 3 * static_cast<size_t>(pages)) * 4; }

cudaError_t launch_compact(const CompactArgs &a, cudaStream_t stream) {
  compact_plan_kernel<<<1, plan_threads(a.c.pages, 1), 0, stream>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_after(compact_move_kernel, dim3(kSms * 8), kThreads, 0, stream, a);
}

}  // namespace bsa
