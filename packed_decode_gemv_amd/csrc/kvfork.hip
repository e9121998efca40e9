// Forks of cached sequences (meaning in vbq.h): two launches, or one for small calls.
//
// k_kv4_fork_plan: its first workgroup counts each old sequence's continuations and
// finds the first of them, counts the pages that every new sequence needs, lists the
// part pages to copy and the lowest free pages, as many as are needed; the others copy
// the reference counts. Which page a sequence gets follows from the numbers alone: the
// i-th page needed, in the order of sequences and their entries, is the i-th free one.
//
// k_kv4_fork: for every new sequence its row of the table, its length and its pages'
// counts, for every old one what its row's pages lose or gain, and by workgroups of
// their own the listed copies. Counts are sums of whole numbers by atomics, the same in
// any order. Pages that are free before the call alone are given out, so no page that is
// read is written.
//
// 512 sequences of 4001 tokens, 8 heads of 128 (26 MB of part pages, read and written):
// the plan 6.4 us, a chain of dependent look-ups and scans by one workgroup, the rest 11.0,
// copies at 4.8 TB/s. One sequence to eight: 5.0 and 3.6 us, look-ups alone. (Few pages in
// reserve each; for many see kept_behind.)
//
// k_kv4_fork_small: where the plan is short every workgroup makes it by itself, so that
// none waits for another's and one launch does. Counts are then summed in LDS, a slice of
// the pages a workgroup. In one and in two launches (us, in a graph; from Python 10.5 and
// 13.1): 1 sequence of 577 tokens to 8, 12 heads of 64, 200 pages 6.6 and 8.1, 60000 pages
// 7.3 and 8.3; 8 of 2000 to 8, 8 heads of 128 4.8 and 6.3; 16 of 1000 to 64 8.7 and 9.0; 64 to
// 64 of 1000 6.0 and 6.7, of 4000 (4032 entries) 7.0 and 6.8; 128 of 2000 7.5 and 6.8; 1 of 250
// to 128 11.3 and 10.1.
#include "kv4.h"

namespace vbq {
namespace {

constexpr int kPlan = 1024;                  // threads of the planning workgroup
constexpr int kPlanKids = 4096;              // old sequences that it counts in LDS
constexpr int kScan = 16;                    // counts that a thread looks at, at a time
// Of small calls: sequences, entries of their rows, pages; of a workgroup's counts; workgroups that copy.
constexpr int kSmallBatch = 64, kSmallRows = 4096, kSmallPages = 65536, kSmallCounts = 4096, kSmallCopiers = 192;

// Of a new sequence: what it goes on from.
struct Parent {
  int p;             // -1: nothing
  int32_t len, whole, have;   // tokens, whole pages, pages
  int64_t need;      // pages with those reserved
  bool bad_len;      // something does not fit
  int32_t part;      // the entry behind the whole pages (of the table's row), -1: no page
  bool part_mine;    // that nothing else names
};
__device__ inline Parent parent_of(const KvFork& f, int b) {
  Parent r;
  r.p = f.parents[b];
  r.len = r.whole = r.have = 0;
  r.bad_len = false;
  int64_t more = f.reserve ? f.reserve[b] : 0;
  if (more < 0) {
    r.bad_len = true;
    more = 0;
  }
  if (r.p >= f.batch_in) r.bad_len = true;
  if (r.p < 0 || r.p >= f.batch_in) r.p = -1;
  const int shift = f.cache.block_shift + 5;
  if (r.p >= 0) {
    const int32_t len = f.lens_in[r.p];
    if (len < 0 || (int64_t)len > ((int64_t)f.width << shift)) {
      r.bad_len = true;
      r.p = -1;
    } else {
      r.len = len;
      r.whole = len >> shift;
      r.have = (int)(((int64_t)len + (1 << shift) - 1) >> shift);
    }
  }
  r.need = (r.len + more + (1 << shift) - 1) >> shift;
  if (r.need > f.width) {
    r.bad_len = true;
    r.need = f.width;
  }
  r.part = -1;
  if (r.p >= 0 && r.whole < r.need) r.part = f.table_in[(int64_t)r.p * f.width + r.whole];
  if ((uint32_t)r.part >= (uint32_t)f.cache.n_pages) r.part = -1;
  r.part_mine = r.part >= 0 && f.refs_in[r.part] == 1;
  return r;
}
// Whether the first continuation keeps entry j (from the part page on) of its parent's row.
__device__ inline bool keeps(const KvFork& f, int p, int j, int32_t& page) {
  page = f.table_in[(int64_t)p * f.width + j];
  return (uint32_t)page < (uint32_t)f.cache.n_pages && f.refs_in[page] == 1;
}

// Inclusive sum over the workgroup; total to every thread. sums: a place a wavefront.
// (WAVES 1: over a wavefront by itself.)
template <int WAVES>
__device__ inline int group_scan(int v, int* sums, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
  if constexpr (WAVES == 1) {
    total = __builtin_amdgcn_readlane(v, 63);
    return v;
  }
  if (lane == 63) sums[wave] = v;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const int s = sums[w];
    before += w < wave ? s : 0;
    total += s;
  }
  __syncthreads();
  return v + before;
}

// How many of `n` entries of old row p, from j0 on, a first continuation keeps (n 0: none).
// The wavefront's lanes each take their own, a look-up after the other (0.17 us an entry),
// or, where the longest are many more than the lanes' share of all, take them in turn (entry
// i of the lanes' one after the other), 512 a step of about 2.5 us. 1 sequence to 8 with pages
// kept for 8, 40, 128 and 1000 entries, each lane its own and shared out, us: 8.5 14.0 28.5 176
// and - 10.0 10.1 20.4; 64 to 64 with 40 each 16.4 and 24.6, 512 to 512 with 64 each 36.3 and 39.4.
constexpr int kFewEntries = 8;
__device__ inline int kept_behind(const KvFork& f, int p, int j0, int n) {
  int kept = 0, total = 0, upto = 0;
  bool share = __any(n > kFewEntries);
  if (share) {
    upto = group_scan<1>(n, nullptr, total);
    share = __any(n > kFewEntries + total / 32);
  }
  if (!share) {
    for (int i = 0, page; i < n; ++i) kept += keeps(f, p, j0 + i, page);
    return kept;
  }
  constexpr int AT_ONCE = 8;
  const int lane = threadIdx.x & 63, before = upto - n;
  for (int i0 = 0; i0 < total; i0 += 64 * AT_ONCE) {
    int32_t page[AT_ONCE];
#pragma unroll
    for (int c = 0; c < AT_ONCE; ++c) {
      const int i = i0 + 64 * c + lane;
      int whose = 0;   // lanes whose entries end at i or before
#pragma unroll
      for (int d = 32; d; d >>= 1) whose += __shfl(upto, whose + d - 1, 64) <= i ? d : 0;
      const int row = __shfl(p, whose, 64), j = __shfl(j0 - before, whose, 64) + i;
      page[c] = i < total ? f.table_in[(int64_t)row * f.width + j] : -1;
    }
    bool keep[AT_ONCE];
#pragma unroll
    for (int c = 0; c < AT_ONCE; ++c) keep[c] = (uint32_t)page[c] < (uint32_t)f.cache.n_pages && f.refs_in[page[c]] == 1;
#pragma unroll
    for (int c = 0; c < AT_ONCE; ++c) {
      const uint64_t who = __ballot(keep[c]);
      const int from = max(before - (i0 + 64 * c), 0), to = min(upto - (i0 + 64 * c), 64);   // the lane's of these 64
      if (from < to) kept += __builtin_popcountll((who >> from) & (~0ull >> (64 - (to - from))));
    }
  }
  return kept;
}

// Places for what the planning workgroup finds (see KvFork), its counts in LDS or not.
struct Plan {
  int *first, *kids, *sums, *copied;
  int4* copies;
  int32_t *offset, *free;
};
// Continuations, pages, copies and free pages; the first `found` of the pages `wanted`
// are there. Flags are set where `tells`.
template <bool IN_LDS>
__device__ inline void plan(const KvFork& f, const Plan& at, bool tells, int& found, int64_t& wanted) {
  const int tid = (int)threadIdx.x;
  if (tid == 0) *at.copied = 0;
  int* const first = at.first;
  int* const kids = at.kids;
  auto get = [](int* p) { return IN_LDS ? *p : __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
  auto put = [](int* p, int v) {
    if (IN_LDS) *p = v;
    else __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  for (int p = tid; p < f.batch_in; p += kPlan) {
    put(first + p, INT32_MAX);
    put(kids + p, 0);
  }
  // Free pages among the thread's first counts, on their way with the rest.
  auto free_at = [&](int64_t at) {
    uint32_t free = 0;
#pragma unroll
    for (int i = 0; i < kScan; i += 4) {
      if (at + i + 4 <= f.cache.n_pages) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(f.refs_in + at + i);
#pragma unroll
        for (int c = 0; c < 4; ++c) free |= (v[c] == 0 ? 1u : 0u) << (i + c);
      } else {
        for (int c = 0; c < 4; ++c)
          if (at + i + c < f.cache.n_pages) free |= (f.refs_in[at + i + c] == 0 ? 1u : 0u) << (i + c);
      }
    }
    return free;
  };
  Parent mine;
  if (tid < f.batch_out) mine = parent_of(f, tid);
  const uint32_t first_free = free_at((int64_t)tid * kScan);
  __builtin_amdgcn_s_waitcnt(VBQ_VMCNT_IMM(0));   // (device-scope stores are where the atomics see them)
  __syncthreads();
  for (int b = tid; b < f.batch_out; b += kPlan) {
    const Parent r = b < kPlan ? mine : parent_of(f, b);
    if (r.bad_len && tells) kv_flag(f.cache, VBQ_KV4_FLAG_LENGTH);
    if (r.p < 0) continue;
    __hip_atomic_fetch_min(first + r.p, b, __ATOMIC_RELAXED, IN_LDS ? __HIP_MEMORY_SCOPE_WORKGROUP : __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_fetch_add(kids + r.p, 1, __ATOMIC_RELAXED, IN_LDS ? __HIP_MEMORY_SCOPE_WORKGROUP : __HIP_MEMORY_SCOPE_AGENT);
  }
  __builtin_amdgcn_s_waitcnt(VBQ_VMCNT_IMM(0));
  __syncthreads();
  // Pages that each new sequence needs, and how many those before it do.
  wanted = 0;
  for (int b0 = 0; b0 < f.batch_out; b0 += kPlan) {
    const int b = b0 + tid;
    int n = 0, blocks = 0, part = -1, p = 0, behind = 0, rest = 0;
    bool is_first = false;
    if (b < f.batch_out) {
      const Parent r = b < kPlan ? mine : parent_of(f, b);
      is_first = r.p >= 0 && get(first + r.p) == b;
      n = (int)r.need - r.whole;
      if (n < 0) n = 0;
      if (r.have > r.whole) {   // a part page: copied unless it is kept
        part = r.part;
        if (part >= 0) blocks = ((r.len & ((kKvBlock << f.cache.block_shift) - 1)) + kKvBlock - 1) / kKvBlock;
      }
      if (is_first) {
        if (r.part_mine) {
          n -= 1;
          blocks = 0;
        }
        p = r.p;
        behind = r.whole + 1;
        rest = max((int)r.need - behind, 0);
      }
    }
    n -= kept_behind(f, p, behind, rest);
    int total;
    const int upto = group_scan<kPlan / 64>(n, at.sums, total);
    // (more than there are pages is cut off: those beyond find none)
    if (b < f.batch_out) {
      const int64_t before = wanted + (upto - n);
      const int from = (int)(before < f.cache.n_pages ? before : f.cache.n_pages);
      at.offset[b] = from | (is_first ? INT32_MIN : 0);
      // A wavefront's copies are listed in the order of its lanes. That of the wavefronts is
      // open, so lists that several workgroups make, each its own, are of one wavefront's.
      const uint64_t who = __ballot(blocks != 0);
      if (blocks) {
        const int lead = __builtin_ctzll(who), n_before = lanes_below(who);
        int place = 0;
        if (n_before == 0)
          place = __hip_atomic_fetch_add(at.copied, __builtin_popcountll(who), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        at.copies[__builtin_amdgcn_readlane(place, lead) + n_before] = int4{part, from, blocks, 0};
      }
    }
    wanted += total;
  }
  // The lowest free pages.
  found = 0;
  const int want = (int)(wanted < f.cache.n_pages ? wanted : f.cache.n_pages);
  for (int64_t base = 0; base < f.cache.n_pages && found < want; base += kPlan * kScan) {
    const int64_t page = base + (int64_t)tid * kScan;
    uint32_t free = base ? free_at(page) : first_free;
    int total;
    int place = found + group_scan<kPlan / 64>(__builtin_popcount(free), at.sums, total) - __builtin_popcount(free);
    for (; free; free &= free - 1, ++place)
      if (place < want) at.free[place] = (int)(page + __builtin_ctz(free));
    found += total;
  }
  found = found < want ? found : want;
  __syncthreads();
  if (tells && tid == 0 && found < wanted) kv_flag(f.cache, VBQ_KV4_FLAG_FULL);
}

// The counts as they were, by workgroup `group` of `groups`.
__device__ inline void keep_counts(const KvFork& f, int64_t group, int64_t groups) {
  const int64_t n = f.cache.n_pages;
  for (int64_t i = (group * kPlan + threadIdx.x) * 4; i < n; i += groups * kPlan * 4) {
    if (i + 4 <= n) *reinterpret_cast<u32x4*>(f.refs_out + i) = *reinterpret_cast<const u32x4*>(f.refs_in + i);
    else
      for (int64_t e = i; e < n; ++e) f.refs_out[e] = f.refs_in[e];
  }
}

constexpr int kCopyAtOnce = 4;   // loads of a thread

// Pieces of the copies, by workgroup `group` of `groups`.
template <int THREADS>
__device__ inline void copy_parts(const KvFork& f, const int4* copies, int n, const int32_t* free, int found, uint32_t group,
                                  uint32_t groups) {
  const int heads = f.cache.heads, unit = kKvGroupBytes * f.cache.groups / 16;   // (of 16 bytes)
  const int stride = unit << f.cache.block_shift;   // between heads
  constexpr int PIECE = THREADS * kCopyAtOnce;
  const int pieces = (stride * heads + PIECE - 1) / PIECE;   // of a whole page
  const int64_t all = (int64_t)n * pieces;
  for (int64_t w = group; w < all; w += groups) {
    const int4 copy = copies[w / pieces];
    const int run = copy.z * unit, end = run * heads, i0 = (int)(w % pieces) * PIECE + (int)threadIdx.x;
    if (copy.y >= found || i0 - (int)threadIdx.x >= end) continue;
    const u32x4* const src = reinterpret_cast<const u32x4*>(kv_block(f.cache, f.cache.groups, (uint32_t)copy.x, 0, 0));
    u32x4* const dst = reinterpret_cast<u32x4*>(kv_block(f.cache, f.cache.groups, (uint32_t)free[copy.y], 0, 0));
    u32x4 v[kCopyAtOnce];
    int o[kCopyAtOnce];
#pragma unroll
    for (int c = 0; c < kCopyAtOnce; ++c) {
      const int i = i0 + c * THREADS;
      o[c] = i < end ? i / run * (stride - run) + i : -1;
      if (o[c] >= 0) v[c] = src[o[c]];
    }
#pragma unroll
    for (int c = 0; c < kCopyAtOnce; ++c)
      if (o[c] >= 0) dst[o[c]] = v[c];
  }
}

// New sequence b: its row, its length, and (COUNTS) what its pages' counts gain.
template <int THREADS, bool COUNTS>
__device__ inline void new_row(const KvFork& f, int b, int off, const int32_t* free, int found, int* sums, int tid) {
  const int32_t n_pages = f.cache.n_pages;
  const Parent r = parent_of(f, b);
  const bool first = off < 0;
  int at = off & INT32_MAX;   // the next page taken
  const int32_t* const from = f.table_in + (int64_t)(r.p < 0 ? 0 : r.p) * f.width;
  if (tid == 0) f.lens_out[b] = r.len;
  int32_t* const to = f.table_out + (int64_t)b * f.width;
  for (int j = tid; j < r.whole; j += THREADS) {
    const int32_t e = from[j];
    const bool ok = (uint32_t)e < (uint32_t)n_pages;
    if (!ok) kv_flag(f.cache, VBQ_KV4_FLAG_PAGE);
    to[j] = ok ? e : -1;
  }
  for (int j0 = r.whole; j0 < (int)r.need; j0 += THREADS) {
    const int j = j0 + tid;
    bool keep = false, fresh = false;
    int32_t e = -1;
    if (j < (int)r.need) {
      if (j < r.have && (uint32_t)from[j] >= (uint32_t)n_pages) kv_flag(f.cache, VBQ_KV4_FLAG_PAGE);
      keep = first && keeps(f, r.p, j, e);
      fresh = !keep;
    }
    int total;
    const int place = at + group_scan<THREADS / 64>(fresh ? 1 : 0, sums, total) - 1;
    if (fresh) e = place < found ? free[place] : -1;
    if (j < (int)r.need) {
      to[j] = e;
      if (COUNTS && e >= 0) __hip_atomic_fetch_add(f.refs_out + e, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    at += total;
  }
  for (int j = (int)(r.need > r.whole ? r.need : r.whole) + tid; j < f.width; j += THREADS) to[j] = -1;
}

template <bool IN_LDS>
__global__ __launch_bounds__(kPlan) void k_kv4_fork_plan(KvFork f) {
  const int tid = (int)threadIdx.x;
  if (blockIdx.x) {
    keep_counts(f, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  __shared__ int lds_first[IN_LDS ? kPlanKids : 1], lds_kids[IN_LDS ? kPlanKids : 1];
  __shared__ int sums[kPlan / 64];
  __shared__ int copied;
  int found;
  int64_t wanted;
  plan<IN_LDS>(f, Plan{IN_LDS ? lds_first : f.first, IN_LDS ? lds_kids : f.kids, sums, &copied, f.copies, f.offset, f.free},
               true, found, wanted);
  if (IN_LDS)
    for (int p = tid; p < f.batch_in; p += kPlan) f.kids[p] = lds_kids[p];
  if (tid == 0) {
    f.head[0] = found;
    f.head[1] = copied;
  }
}

constexpr int kForkThreads = 256;

__global__ __launch_bounds__(kForkThreads) void k_kv4_fork(KvFork f) {
  __shared__ int sums[kForkThreads / 64];
  const int tid = (int)threadIdx.x;
  if (blockIdx.x < f.copiers) {
    copy_parts<kForkThreads>(f, f.copies, f.head[1], f.free, f.head[0], blockIdx.x, f.copiers);
    return;
  }
  const uint32_t block = blockIdx.x - f.copiers;
  if (block >= (uint32_t)f.batch_out) {
    // an old sequence: its row is gone, its whole pages go to its continuations
    const int p = (int)(block - (uint32_t)f.batch_out), kids = f.kids[p];
    const int32_t whole = kids ? f.lens_in[p] >> (f.cache.block_shift + 5) : 0;
    for (int j = tid; j < f.width; j += kForkThreads) {
      const int32_t page = f.table_in[(int64_t)p * f.width + j];
      const int d = (j < whole ? kids : 0) - 1;
      if ((uint32_t)page < (uint32_t)f.cache.n_pages) {
        if (d) __hip_atomic_fetch_add(f.refs_out + page, d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      } else if (page != -1) {
        kv_flag(f.cache, VBQ_KV4_FLAG_PAGE);
      }
    }
  } else {
    new_row<kForkThreads, true>(f, (int)block, f.offset[block], f.free, f.head[0], sums, tid);
  }
}

// Small calls: every workgroup plans by itself, then takes a share of the counts, of the
// rows, or of the copies.
__global__ __launch_bounds__(kPlan) void k_kv4_fork_small(KvFork f) {
  static_assert(kSmallBatch <= 64, "the copies are listed by one wavefront, the same in every workgroup");
  __shared__ int first[kSmallBatch], kids[kSmallBatch], sums[kPlan / 64], copied;
  __shared__ int4 copies[kSmallBatch];
  __shared__ int32_t offset[kSmallBatch], free[kSmallRows], counts[kSmallCounts];
  __shared__ int2 old[kSmallBatch];   // of an old sequence with continuations: whole pages, pages that the first has
  const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int counters = (f.cache.n_pages + kSmallCounts - 1) / kSmallCounts, block = (int)blockIdx.x;
  const int rows = (f.batch_out + kPlan / 64 - 1) / (kPlan / 64);
  const bool counts_here = block < counters;
  const int page0 = counts_here ? block * kSmallCounts : 0, pages = min(f.cache.n_pages - page0, kSmallCounts);
  if (counts_here)
    for (int i = tid; i < pages; i += kPlan) counts[i] = f.refs_in[page0 + i];
  int found;
  int64_t wanted;
  plan<true>(f, Plan{first, kids, sums, &copied, copies, offset, free}, block == 0, found, wanted);
  if (block >= counters + rows) {
    copy_parts<kPlan>(f, copies, copied, free, found, (uint32_t)(block - counters - rows), gridDim.x - (uint32_t)(counters + rows));
    return;
  }
  if (!counts_here) {   // a sequence a wavefront
    const int b = (block - counters) * (kPlan / 64) + wave;
    if (b < f.batch_out) new_row<64, false>(f, b, offset[b], free, found, sums, lane);
    return;
  }
  // What the old rows' entries lose and gain (those that the first continuation keeps stay), and the pages taken.
  if (tid < f.batch_in) {
    const int b = first[tid];
    const Parent r = parent_of(f, b == INT32_MAX ? 0 : b);
    old[tid] = b == INT32_MAX ? int2{0, 0} : int2{r.whole, (int)r.need};
  }
  __syncthreads();
  for (int i = tid; i < f.batch_in * f.width; i += kPlan) {
    const int p = i / f.width, j = i - p * f.width;
    const int32_t page = f.table_in[i];
    if ((uint32_t)page >= (uint32_t)f.cache.n_pages) {
      if (page != -1 && block == 0) kv_flag(f.cache, VBQ_KV4_FLAG_PAGE);
      continue;
    }
    if ((uint32_t)(page - page0) >= (uint32_t)pages) continue;
    const int d = (j < old[p].x ? kids[p] : j < old[p].y && f.refs_in[page] == 1 ? 1 : 0) - 1;
    if (d) __hip_atomic_fetch_add(counts + (page - page0), d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  }
  for (int i = tid; i < found; i += kPlan) {
    const int page = free[i] - page0;
    if ((uint32_t)page < (uint32_t)pages)
      __hip_atomic_fetch_add(counts + page, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  }
  __syncthreads();
  for (int i = tid; i < pages; i += kPlan) f.refs_out[page0 + i] = counts[i];
}

}  // namespace

hipError_t launch_kv4_fork(const KvFork& f, hipStream_t s) {
  const int64_t page = (int64_t)f.cache.heads * f.cache.groups * kKvGroupBytes << f.cache.block_shift;
  if (f.batch_in <= kSmallBatch && f.batch_out <= kSmallBatch && (int64_t)f.batch_out * f.width <= kSmallRows &&
      (int64_t)f.batch_in * f.width <= kSmallRows && f.cache.n_pages <= kSmallPages) {
    const int64_t pieces = f.batch_out * ((page + kPlan * kCopyAtOnce * 16 - 1) / (kPlan * kCopyAtOnce * 16));
    const int64_t others = (f.cache.n_pages + kSmallCounts - 1) / kSmallCounts + (f.batch_out + kPlan / 64 - 1) / (kPlan / 64);
    k_kv4_fork_small<<<dim3((uint32_t)(others + (pieces < kSmallCopiers ? pieces : kSmallCopiers))), kPlan, 0, s>>>(f);
    return hipGetLastError();
  }
  const int64_t copies = (f.cache.n_pages + kPlan * 4 - 1) / (kPlan * 4);
  const dim3 plan_grid((uint32_t)(1 + (copies < 64 ? copies : 64)));
  if (f.batch_in <= kPlanKids) k_kv4_fork_plan<true><<<plan_grid, kPlan, 0, s>>>(f);
  else k_kv4_fork_plan<false><<<plan_grid, kPlan, 0, s>>>(f);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // (a page is copied for every new sequence, at most; more workgroups than fill the chip take turns)
  const int64_t pieces = f.batch_out * ((page + kForkThreads * kCopyAtOnce * 16 - 1) / (kForkThreads * kCopyAtOnce * 16));
  KvFork k = f;
  k.copiers = (uint32_t)(pieces < 2048 ? pieces : 2048);
  const dim3 grid(k.copiers + (uint32_t)(f.batch_out + f.batch_in));
  k_kv4_fork<<<grid, kForkThreads, 0, s>>>(k);
  return hipGetLastError();
}

}  // namespace vbq
