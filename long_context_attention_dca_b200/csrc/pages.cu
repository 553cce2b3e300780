// Pages of a cache: which slot holds which page, and the moves that follow.
//
// A pool is num_blocks pages; slot b of the block table [B][max_blocks] lists
// the pages of its sequence; refs[p] counts the table entries that name page p
// (plus whatever the caller added to keep a page).  Both operations are
// functions of that state with one result: pages are taken lowest index first,
// slots served in order, so neither the launch shape nor the order of atomics
// shows in the outputs.
//
// Each runs as two kernels.  The plan is integer work over B * max_blocks
// entries and num_blocks counts with a handful of dependent phases.  A state
// that fits one CTA's shared memory is planned there by that CTA; a larger one
// by a cluster of 8 CTAs in global memory, whose hardware barrier separates the
// phases.  The copies move the bytes, a chunk a block at a time, from a list
// whose length stays on the device; they are bound by memory bandwidth.
#include "dca_common.cuh"
#include "dca_kernels.cuh"

namespace dca {
namespace pages {

constexpr int kPlanThreads = 1024;
constexpr int kNone = 0x7FFFFFFF;

// C CTAs plan together.  Working arrays written by one and read by another are
// read past the L1 cache; a CTA alone has them in shared memory.
template <int C>
__device__ __forceinline__ void phase_end() {
  if (C == 1) {
    __syncthreads();
  } else {
    __threadfence();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}
template <int C>
__device__ __forceinline__ int get(const int* p) {
  return C == 1 ? *p : __ldcg(p);
}
__device__ __forceinline__ int pages_of(int n, int R) {  // n >= 0, R <= 2^30
  return (int)(((unsigned)n + (unsigned)R - 1u) / (unsigned)R);
}
// The entries of the block table dealt to the threads, every step-th one to each,
// as (slot, place in it): one division to begin with, none to go on.  Taken N at
// a time, whose loads are in flight together; an entry past the end is the first
// one, not live.  Two at a time in shared memory (191 pages: 5.5 us against 5.6
// with four), four in global memory (271887 ints: 50 us against 52 with two).
template <int C>
constexpr int kBatchOf = C == 1 ? 2 : 4;
struct Entries {
  int b, i, e, B, max_blocks, step, slots, places;
  __device__ Entries(int first, int step_, int B_, int max_blocks_)
      : b(first / max_blocks_),
        i(first % max_blocks_),
        e(first),
        B(B_),
        max_blocks(max_blocks_),
        step(step_),
        slots(step_ / max_blocks_),
        places(step_ % max_blocks_) {}
};
template <int N>
struct Batch {
  int b[N], i[N], e[N];
  bool live[N];
  __device__ __forceinline__ explicit Batch(Entries& at) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      live[u] = at.b < at.B;
      b[u] = live[u] ? at.b : 0;
      i[u] = live[u] ? at.i : 0;
      e[u] = live[u] ? at.e : 0;
      at.e += at.step;
      at.b += at.slots;
      at.i += at.places;
      if (at.i >= at.max_blocks) {
        at.i -= at.max_blocks;
        ++at.b;
      }
    }
  }
};

// Exclusive prefix sums of one value a thread over the block; `total` gets the sum.
// One barrier each: every warp adds up the warps' sums for itself, and two sets of
// them take turns.
constexpr int kScanInts = 2 * 32;
struct Scan {
  int* sums;  // [kScanInts], shared
  int turn;
  __device__ explicit Scan(int* p) : sums(p), turn(0) {}
  __device__ __forceinline__ int operator()(int v, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int x = inclusive(v, lane);
    if (lane == 31) sums[turn + warp] = x;
    __syncthreads();
    const int all = inclusive(sums[turn + lane], lane);
    turn ^= 32;
    total = __shfl_sync(0xFFFFFFFFu, all, 31);
    const int before = __shfl_sync(0xFFFFFFFFu, all, warp ? warp - 1 : 0);
    return (warp ? before : 0) + x - v;
  }
  __device__ static __forceinline__ int inclusive(int x, int lane) {
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, sh);
      if (lane >= sh) x += y;
    }
    return x;
  }
};

// Part of 0 .. n-1 that CTA `rank` scans: contiguous, so that a rank within the
// part plus the parts before it is a rank in the whole.
struct Part {
  int begin, end;
};
template <int C>
__device__ __forceinline__ Part part_of(int n, int rank) {
  const int per = (int)(((long long)n + C - 1) / C);
  const long long a = (long long)per * rank;
  return Part{(int)min(a, (long long)n), (int)min(a + per, (long long)n)};
}

struct Work {  // all int32
  int* out;     // [64]: 0 copies.  Always in the workspace, as the copy list:
  int* from;    // [max(num_blocks, B)] source page
  int* to;      //                      target page
  int* rows;    //                      rows to copy
  int* head;    // [64]: 0 faults, 1 copies, 2 pages wanted; 8.. per-CTA sums
  int* count;   // [num_blocks] references while the plan runs
  int* owner;   // [num_blocks] slot that keeps a partial page; a page's new index
  int* list;    // [num_blocks] free pages or holes, ascending
  int* table;   // [B * max_blocks] the table as it came
  int* slots;   // [6][B] see slot()
};
constexpr int kHead = 64;

size_t list_ints(int B, int num_blocks) {
  return kHead + 3 * (size_t)(num_blocks > B ? num_blocks : B);
}
__host__ __device__ inline size_t plan_ints(int B, int max_blocks, int num_blocks) {
  return kHead + 3 * (size_t)num_blocks + (size_t)B * max_blocks + 6 * (size_t)B;
}
size_t work_ints(int B, int max_blocks, int num_blocks) {
  return list_ints(B, num_blocks) + plan_ints(B, max_blocks, num_blocks);
}
// A plan of this many ints or fewer runs in one CTA's shared memory (200 KB).
// Alone against a cluster in global memory, us (remap / compact): 1037 ints 5.1 /
// 4.6 against 16.5 / 12.6, 16017 ints 10.0 / 9.1 against 18.1 / 13.2, 38073 ints
// 17.4 / 15.1 against 21.0 / 14.9: the compaction's two forms meet there, the remap's
// later.
constexpr size_t kAloneInts = 50000;

__host__ __device__ inline void carve_plan(Work& w, int* p, int B, int max_blocks,
                                           int num_blocks) {
  w.head = p;
  w.count = w.head + kHead;
  w.owner = w.count + num_blocks;
  w.list = w.owner + num_blocks;
  w.table = w.list + num_blocks;
  w.slots = w.table + (size_t)B * max_blocks;
}
Work carve(void* ws, int B, int max_blocks, int num_blocks) {
  const size_t m = (size_t)(num_blocks > B ? num_blocks : B);
  Work w;
  w.out = static_cast<int*>(ws);
  w.from = w.out + kHead;
  w.to = w.from + m;
  w.rows = w.to + m;
  carve_plan(w, w.rows + m, B, max_blocks, num_blocks);
  return w;
}

// What becomes of a slot, worked out once, by a thread each: keep = min(old_len[src],
// new_len) rows of old slot src (none for -1) are `full` whole pages and `rest`
// rows of the next.  Six arrays of the slots:
enum {
  kSrc,
  kFull,
  kRest,   // later 0 where the slot keeps the partial page itself: nothing to copy
  kPages,  // of the new length
  kUsed,   // of the old length; later the entries that stay, full pages and partial one
  kFresh,  // entry i beyond those is the new page list[kFresh + i]
};
__device__ __forceinline__ int* slot(const Work& w, int what, int B, int b) {
  return w.slots + (size_t)what * B + b;
}
// The table as it came into the working copy: independent loads, eight in flight
// a thread, since nothing else hides their latency.
__device__ __forceinline__ void stage(const int* from, int* to, int n, int first, int step) {
  for (long long e = first; e < n; e += 8ll * step) {
    int v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      v[u] = e + (long long)u * step < n ? from[e + (long long)u * step] : 0;
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (e + (long long)u * step < n) to[e + (long long)u * step] = v[u];
  }
}

// Full pages are shared.  A partial last page goes to the lowest slot that wants
// it unless it is still held elsewhere; every other slot gets a copy of its rows.
// The entries of the table are dealt to the threads one by one, whatever their
// slots: 192 slots of 35 entries and 2715 pages take 10.3 us, against 13.7 with a
// warp a slot; 2000 slots of 60 and 46629 pages 50 against 57.
template <int C>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kPlanThreads, 1) remap_plan(
    const int* __restrict__ src, const int* __restrict__ old_len,
    const int* __restrict__ new_len, const int* table_in, int* table_out, const int* refs_in,
    int* refs_out, int* __restrict__ info, int B, int max_blocks, int num_blocks, int R,
    Work w) {
  __shared__ int sums[kScanInts];
  Scan block_scan(sums);
  const int rank = blockIdx.x, tid = threadIdx.x;
  const int gid = rank * kPlanThreads + tid;
  constexpr int kAll = C * kPlanThreads, kBatch = kBatchOf<C>;
  const Entries first(gid, kAll, B, max_blocks);
  extern __shared__ int plan_smem[];
  if (C == 1) carve_plan(w, plan_smem, B, max_blocks, num_blocks);
  cudaTriggerProgrammaticLaunchCompletion();  // the copies may take their places
  const long long cap = (long long)max_blocks * R;
  if (rank == 0 && tid < kHead) w.head[tid] = 0;
  bool bad = false;
  int f = 0, n = 0, o = 0;  // of the thread's first slot, fetched beside the table
  if (gid < B) f = src[gid], n = new_len[gid], o = old_len[gid];
  stage(table_in, w.table, B * max_blocks, gid, kAll);
#pragma unroll 4
  for (int p = gid; p < num_blocks; p += kAll) {
    const int held = refs_in[p];
    w.count[p] = held;
    w.owner[p] = kNone;
    bad |= held < 0;
  }
  for (int b = gid; b < B; b += kAll) {
    if (b != gid) f = src[b], n = new_len[b], o = old_len[b];
    const bool fits = o >= 0 && o <= cap;
    bad |= f < -1 || f >= B || n < 0 || n > cap || !fits;
    const int keep = f < 0 || f >= B ? 0 : max(0, min(old_len[f], n));
    const int full = (int)((unsigned)keep / (unsigned)R);
    *slot(w, kSrc, B, b) = f;
    *slot(w, kFull, B, b) = full;
    *slot(w, kRest, B, b) = keep - full * R;
    *slot(w, kPages, B, b) = pages_of(max(n, 0), R);
    *slot(w, kUsed, B, b) = fits ? pages_of(o, R) : 0;
  }
  phase_end<C>();

  // what the slots hold dropped from the counts; a fault anywhere refuses the
  // whole call
  for (Entries at = first; at.b < B;) {
    const Batch<kBatch> x(at);
    int p[kBatch], used[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      used[u] = get<C>(slot(w, kUsed, B, x.b[u]));
      p[u] = get<C>(w.table + x.e[u]);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (!x.live[u] || x.i[u] >= used[u]) continue;
      if (p[u] < 0 || p[u] >= num_blocks) bad = true;
      else if (atomicSub(w.count + p[u], 1) <= 0) bad = true;  // fewer than name it
    }
  }
  if (bad) atomicExch(w.head, 1);
  phase_end<C>();
  const bool fault = get<C>(w.head) != 0;

  // full pages are shared by every slot that keeps them
  if (!fault) {
    for (Entries at = first; at.b < B;) {
      const Batch<kBatch> x(at);
      int p[kBatch], full[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        full[u] = get<C>(slot(w, kFull, B, x.b[u]));
        p[u] = max(get<C>(slot(w, kSrc, B, x.b[u])), 0) * max_blocks + x.i[u];
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) p[u] = get<C>(w.table + p[u]);
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (x.live[u] && x.i[u] < full[u]) atomicAdd(w.count + p[u], 1);
    }
  }
  phase_end<C>();
  // partial pages that nobody holds any more go to the lowest slot
  auto tail_of = [&](int b) {
    return get<C>(w.table + (size_t)get<C>(slot(w, kSrc, B, b)) * max_blocks +
                  get<C>(slot(w, kFull, B, b)));
  };
  if (!fault) {
    for (int b = gid; b < B; b += kAll) {
      if (get<C>(slot(w, kRest, B, b)) == 0) continue;
      const int p = tail_of(b);
      if (get<C>(w.count + p) == 0) atomicMin(w.owner + p, b);
    }
  }
  phase_end<C>();

  // free pages, each CTA counting its own part
  const Part mine = part_of<C>(num_blocks, rank);
  if (C > 1) {
    int local = 0;
    for (int p = mine.begin + tid; p < mine.end; p += kPlanThreads)
      local += get<C>(w.count + p) == 0 && get<C>(w.owner + p) == kNone;
    int part_free;
    block_scan(local, part_free);
    if (tid == 0) w.head[8 + rank] = part_free;
  }
  // where each slot's new pages start among all new pages
  if (rank == 0) {
    int carry = 0;
    for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
      const int b = b0 + tid;
      int need = 0, stay = 0;
      if (b < B && !fault) {
        stay = get<C>(slot(w, kFull, B, b));
        if (get<C>(slot(w, kRest, B, b)) && get<C>(w.owner + tail_of(b)) == b) {
          ++stay;
          *slot(w, kRest, B, b) = 0;
        }
        need = get<C>(slot(w, kPages, B, b)) - stay;
      }
      int total;
      const int before = block_scan(need, total);
      if (b < B) {
        *slot(w, kUsed, B, b) = stay;
        *slot(w, kFresh, B, b) = carry + before - stay;
      }
      carry += total;
    }
    if (tid == 0) w.head[2] = carry;
  }
  phase_end<C>();

  // free pages in ascending order, and the new counts
  const int need_all = get<C>(w.head + 2);
  int before = 0, free_all = 0;
  if (C > 1) {
    for (int r = 0; r < C; ++r) {
      const int n = get<C>(w.head + 8 + r);
      if (r < rank) before += n;
      free_all += n;
    }
  }
  if (!fault && (C == 1 || need_all <= free_all)) {
    for (int p0 = mine.begin; p0 < mine.end; p0 += kPlanThreads) {
      const int p = p0 + tid;
      int n = 0, free = 0;
      if (p < mine.end) {
        n = get<C>(w.count + p);
        if (get<C>(w.owner + p) != kNone) n = 1;  // kept by one slot
        free = n == 0;
      }
      int total;
      const int at = before + block_scan(free, total);
      if (p < mine.end) {
        if (free) {
          w.list[at] = p;
          n = at < need_all;
        }
        w.count[p] = n;
      }
      before += total;
    }
  }
  if (C == 1) free_all = before;
  if (fault || need_all > free_all) {  // refused: the state as it came
    for (long long e = gid; e < (long long)B * max_blocks; e += kAll)
      table_out[e] = get<C>(w.table + e);
    if (refs_out != refs_in)
      for (int p = gid; p < num_blocks; p += kAll) refs_out[p] = refs_in[p];
    if (gid == 0) {
      info[0] = fault ? kNone : -(need_all - free_all);
      info[1] = w.out[0] = 0;
      if (fault) report_error(kDevBadArg, 209);
    }
    return;
  }
  phase_end<C>();

  for (int b = gid; b < B; b += kAll) {
    const int rest = get<C>(slot(w, kRest, B, b));
    if (rest == 0) continue;
    const int k = atomicAdd(w.head + 1, 1), full = get<C>(slot(w, kFull, B, b));
    w.from[k] = tail_of(b);
    w.to[k] = get<C>(w.list + get<C>(slot(w, kFresh, B, b)) + full);
    w.rows[k] = rest;
  }
  for (int p = gid; p < num_blocks; p += kAll) refs_out[p] = get<C>(w.count + p);
  for (Entries at = first; at.b < B;) {
    const Batch<kBatch> x(at);
    const int* from[kBatch];
    int page[kBatch], pages[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int b = x.b[u], i = x.i[u];
      pages[u] = get<C>(slot(w, kPages, B, b));
      const int src = get<C>(slot(w, kSrc, B, b)), fresh = get<C>(slot(w, kFresh, B, b));
      from[u] = i < get<C>(slot(w, kUsed, B, b)) ? w.table + src * max_blocks + i
                                                 : w.list + (i < pages[u] ? fresh + i : 0);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) page[u] = get<C>(from[u]);
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (x.live[u]) table_out[x.e[u]] = x.i[u] < pages[u] ? page[u] : -1;
  }
  phase_end<C>();
  if (gid == 0) {
    info[0] = free_all - need_all;
    info[1] = w.out[0] = get<C>(w.head + 1);
  }
}

// Pages in use (refs > 0) with an index of n or more, n their number, move to
// the free indexes below n, both in ascending order.
template <int C>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kPlanThreads, 1) compact_plan(
    const int* __restrict__ len, const int* table_in, int* table_out, const int* refs_in,
    int* refs_out, int* __restrict__ moved, int* __restrict__ info, int B, int max_blocks,
    int num_blocks, int R, Work w) {
  __shared__ int sums[kScanInts];
  Scan block_scan(sums);
  const int rank = blockIdx.x, tid = threadIdx.x;
  const int gid = rank * kPlanThreads + tid;
  constexpr int kAll = C * kPlanThreads, kBatch = kBatchOf<C>;
  const Entries first(gid, kAll, B, max_blocks);
  extern __shared__ int plan_smem[];
  if (C == 1) carve_plan(w, plan_smem, B, max_blocks, num_blocks);
  cudaTriggerProgrammaticLaunchCompletion();  // the copies may take their places
  const long long cap = (long long)max_blocks * R;
  const Part mine = part_of<C>(num_blocks, rank);
  if (rank == 0 && tid < 8) w.head[tid] = 0;
  bool bad = false;
  int local = 0;
  for (int b = gid; b < B; b += kAll) {
    const int n = len[b];
    const bool fits = n >= 0 && n <= cap;
    bad |= !fits;
    w.slots[b] = fits ? pages_of(n, R) : 0;
  }
  stage(table_in, w.table, B * max_blocks, gid, kAll);
#pragma unroll 4
  for (int p = mine.begin + tid; p < mine.end; p += kPlanThreads) {
    const int n = refs_in[p];
    w.count[p] = n;
    local += n > 0;
    bad |= n < 0;
  }
  int part_live;
  block_scan(local, part_live);
  if (tid == 0) w.head[8 + rank] = part_live;
  phase_end<C>();
  for (Entries at = first; at.b < B;) {
    const Batch<kBatch> x(at);
    int p[kBatch], n[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      p[u] = x.live[u] && x.i[u] < get<C>(w.slots + x.b[u]) ? get<C>(w.table + x.e[u]) : kNone;
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      n[u] = get<C>(w.count + ((unsigned)p[u] < (unsigned)num_blocks ? p[u] : 0));
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      bad |= x.live[u] && x.i[u] < get<C>(w.slots + x.b[u]) &&
             ((unsigned)p[u] >= (unsigned)num_blocks || n[u] <= 0);
  }
  if (bad) atomicExch(w.head, 1);
  int before = 0, live = 0;
  for (int r = 0; r < C; ++r) {
    const int n = get<C>(w.head + 8 + r);
    if (r < rank) before += n;
    live += n;
  }
  // how many of the pages below n are in use
  local = 0;
  for (int p = mine.begin + tid; p < min(mine.end, live); p += kPlanThreads)
    local += w.count[p] > 0;
  int part_low;
  block_scan(local, part_low);
  if (tid == 0) w.head[16 + rank] = part_low;
  phase_end<C>();
  if (get<C>(w.head)) {
    for (long long e = gid; e < (long long)B * max_blocks; e += kAll)
      table_out[e] = get<C>(w.table + e);
    if (refs_out != refs_in)
      for (int p = gid; p < num_blocks; p += kAll) refs_out[p] = refs_in[p];
    for (int p = gid; p < num_blocks; p += kAll) moved[p] = p;
    if (gid == 0) {
      info[0] = kNone;
      info[1] = w.out[0] = 0;
      report_error(kDevBadArg, 210);
    }
    return;
  }
  int low = 0;
  for (int r = 0; r < C; ++r) low += get<C>(w.head + 16 + r);
  for (int p0 = mine.begin; p0 < mine.end; p0 += kPlanThreads) {
    const int p = p0 + tid;
    const int used = p < mine.end && w.count[p] > 0;
    int total;
    const int at = before + block_scan(used, total);  // pages in use below p
    if (p < mine.end) {
      if (used && p >= live) w.from[at - low] = p;
      if (!used && p < live) w.to[p - at] = p;
    }
    before += total;
  }
  phase_end<C>();
  const int moves = live - low;
  for (int p = gid; p < num_blocks; p += kAll) {
    const int n = get<C>(w.count + p);
    w.owner[p] = moved[p] = n > 0 && p < live ? p : -1;
    refs_out[p] = p < live ? n : 0;  // holes are filled below
  }
  phase_end<C>();
  for (int k = gid; k < moves; k += kAll) {
    const int a = get<C>(w.from + k), z = get<C>(w.to + k);
    w.owner[a] = moved[a] = z;
    refs_out[z] = get<C>(w.count + a);
    w.rows[k] = R;
  }
  phase_end<C>();
  for (Entries at = first; at.b < B;) {
    const Batch<kBatch> x(at);
    int p[kBatch];
    bool used[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      used[u] = x.i[u] < get<C>(w.slots + x.b[u]);
      p[u] = get<C>(w.table + x.e[u]);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) p[u] = get<C>(w.owner + (used[u] ? p[u] : 0));
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (x.live[u]) table_out[x.e[u]] = used[u] ? p[u] : -1;
  }
  if (gid == 0) {
    info[0] = live;
    info[1] = w.out[0] = moves;
  }
}

// Copies of the list, in every pool: the first ceil(rows / unit_rows) units of
// each outer part of a page.  A work item is one chunk of one part; items are
// numbered over the longest possible copy and the ones past a short copy's end
// do nothing.  Bound by memory: compacting 975 MB of bf16 pages (1.95 GB in and
// out) takes 313 us, 6.2 TB/s.  A block finds its pool by a walk over the list, which
// shows only where many pools have few pages to copy: a remap with 3 copies in 64
// bf16 pools (79 MB moved) takes 21 us, plan included, with 64 copies 235 us (1678
// MB); in 256 pools with 3 copies 124 us (315 MB, 48 us at the copy rate).
constexpr int kChunk = 32 << 10;
constexpr int kCopyThreads = 256;

template <int N>
__global__ void __launch_bounds__(kCopyThreads) copy_pages(const __grid_constant__ Pools<N> pools,
                                                           int R, Work w) {
  cudaGridDependencySynchronize();  // the plan's list
  const int n = __ldcg(w.out);
  const long long items = (long long)n * pools.items;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int k = (int)(it / pools.items);
    int rem = (int)(it % pools.items), j = 0;
    while (rem >= pools.p[j].items) rem -= pools.p[j++].items;
    const PoolDesc d = pools.p[j];
    const int part = rem / d.chunks, chunk = rem % d.chunks;
    const int units = (__ldcg(w.rows + k) + d.unit_rows - 1) / d.unit_rows;
    const long long bytes = (long long)units * d.unit_bytes;
    const long long at = (long long)chunk * kChunk;
    if (at >= bytes) continue;
    const long long part_bytes = (long long)(R / d.unit_rows) * d.unit_bytes;
    const size_t a = ((size_t)__ldcg(w.from + k) * d.outer + part) * part_bytes + at;
    const size_t z = ((size_t)__ldcg(w.to + k) * d.outer + part) * part_bytes + at;
    const int words = (int)(min(bytes - at, (long long)kChunk) / 16);
    const uint4* from = reinterpret_cast<const uint4*>(d.base + a);
    uint4* to = reinterpret_cast<uint4*>(d.base + z);
    constexpr int kPer = kChunk / 16 / kCopyThreads;
    uint4 v[kPer];
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int x = threadIdx.x + u * kCopyThreads;
      if (x < words) v[u] = __ldcs(from + x);
    }
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int x = threadIdx.x + u * kCopyThreads;
      if (x < words) __stcs(to + x, v[u]);
    }
  }
}

// `most`: the largest number of copies the plan can ask for.
cudaError_t launch_copies(PoolList& pools, int R, const Work& w, long long most,
                          cudaStream_t stream) {
  pools.items = 0;
  for (int j = 0; j < pools.n; ++j) {
    PoolDesc& d = pools.p[j];
    const long long part = (long long)(R / d.unit_rows) * d.unit_bytes;
    d.chunks = (int)((part + kChunk - 1) / kChunk);
    d.items = d.outer * d.chunks;
    pools.items += d.items;
  }
  if (pools.items == 0 || most == 0) return cudaSuccess;
  // six blocks an SM are resident
  const int grid = most >= 148 * 6 || most * pools.items >= 148 * 6 ? 148 * 6
                                                                   : (int)(most * pools.items);
  // The list travels with the launch, at a cost by its size: two sizes of it.
  if (pools.n <= 16) {
    Pools<16> few;
    few.items = pools.items;
    few.n = pools.n;
    for (int j = 0; j < pools.n; ++j) few.p[j] = pools.p[j];
    return launch_early(copy_pages<16>, dim3(grid), kCopyThreads, stream, few, R, w);
  }
  return launch_early(copy_pages<kMaxPools>, dim3(grid), kCopyThreads, stream, pools, R, w);
}

// Shared memory of a CTA that plans alone, or 0 where the state is too large.
template <typename K>
cudaError_t alone_bytes(K kern, int B, int max_blocks, int num_blocks, size_t& bytes) {
  const size_t ints = plan_ints(B, max_blocks, num_blocks);
  bytes = 0;
  if (ints > kAloneInts) return cudaSuccess;
  bytes = ints * sizeof(int);
  // 48 KB without asking, the kernel's own arrays included
  return bytes + kScanInts * sizeof(int) <= 48 << 10
             ? cudaSuccess
             : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)(kAloneInts * sizeof(int)));
}

}  // namespace pages

size_t pages_workspace_bytes(int B, int max_blocks, int num_blocks) {
  return pages::work_ints(B, max_blocks, num_blocks) * sizeof(int);
}

cudaError_t launch_pages_remap(const int* src, const int* old_len, const int* new_len,
                               const int* table_in, int* table_out, const int* refs_in,
                               int* refs_out, int* info, int B, int max_blocks, int num_blocks,
                               int block_rows, PoolList& pools, void* workspace,
                               cudaStream_t stream) {
  using namespace pages;
  const Work w = carve(workspace, B, max_blocks, num_blocks);
  size_t alone;
  cudaError_t e = alone_bytes(remap_plan<1>, B, max_blocks, num_blocks, alone);
  if (e != cudaSuccess) return e;
  auto plan = alone ? remap_plan<1> : remap_plan<8>;
  plan<<<alone ? 1 : 8, kPlanThreads, alone, stream>>>(
      src, old_len, new_len, table_in, table_out, refs_in, refs_out, info, B, max_blocks,
      num_blocks, block_rows, w);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_copies(pools, block_rows, w, B, stream) : e;
}

cudaError_t launch_pages_compact(const int* len, const int* table_in, int* table_out,
                                 const int* refs_in, int* refs_out, int* moved, int* info, int B,
                                 int max_blocks, int num_blocks, int block_rows, PoolList& pools,
                                 void* workspace, cudaStream_t stream) {
  using namespace pages;
  const Work w = carve(workspace, B, max_blocks, num_blocks);
  size_t alone;
  cudaError_t e = alone_bytes(compact_plan<1>, B, max_blocks, num_blocks, alone);
  if (e != cudaSuccess) return e;
  auto plan = alone ? compact_plan<1> : compact_plan<8>;
  plan<<<alone ? 1 : 8, kPlanThreads, alone, stream>>>(
      len, table_in, table_out, refs_in, refs_out, moved, info, B, max_blocks, num_blocks,
      block_rows, w);
  e = cudaGetLastError();
  return e == cudaSuccess ? launch_copies(pools, block_rows, w, num_blocks / 2, stream) : e;
}

}  // namespace dca
