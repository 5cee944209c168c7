// kv_pages.hip — the pages of a cache: copied, given back, forked, moved
// together.
//
// What bounds them: the bytes of the pages that move, read once and written
// once; the rest is a few passes over the reference counts and tables. What
// the host cannot know (which pages are free, how many move) is worked out on
// the device: one workgroup writes a list of (from, to) pages into the
// workspace, and a second launch whose size the host bounds moves them. Every
// allocation takes the lowest free pages in the order of the request, found by
// a scan, so results do not depend on timing.
//
// Measured: 2.1 GB read and written by a compaction of 8 layers x 8192 pages of
// 32 KB 430 us, 4.9 TB/s, a large copy's rate; its list 5.4 us. 64 beams freed
// and forked 17 us: 2.6 + 8.1 (the list) + 5.5.
#include <algorithm>

#include "kv_device.h"
#include "kv_launch.h"

namespace xq {
namespace {

constexpr int kThreads = 256;
constexpr int kListThreads = 1024;
constexpr int kRun = 8;  // pages in a row that a thread of the lists takes
// The first bytes of a workspace are where other calls keep counters that
// have to stay zero.
constexpr size_t kCounterRegion = 96 * 1024;

struct PageArgs {
  uint8_t* base[2];                           // k, v
  int64_t layer[2], page[2], head[2], tok[2]; // bytes
  int64_t rows_bytes;                         // dim in bytes
  int64_t whole;                              // bytes of a page of one layer, when it is one run; else 0
  int layers, kv_heads, page_tokens, pages;
  int pieces;                                 // workgroups that share a page of one layer
};

// One page of one layer of k or v, or a part of it: 16-byte words.
__device__ __forceinline__ void copy_page(const PageArgs& a, int which, int layer, int piece,
                                          int64_t from, int64_t to) {
  const uint8_t* src = a.base[which] + layer * a.layer[which] + from * a.page[which];
  uint8_t* dst = a.base[which] + layer * a.layer[which] + to * a.page[which];
  if (a.whole) {
    const int64_t words = a.whole / 16;
    const u32x4* s = reinterpret_cast<const u32x4*>(src);
    u32x4* d = reinterpret_cast<u32x4*>(dst);
    const int64_t step = static_cast<int64_t>(kThreads) * a.pieces;
    int64_t i = static_cast<int64_t>(piece) * kThreads + threadIdx.x;
    for (; i + 3 * step < words; i += 4 * step) {
      const u32x4 w0 = s[i], w1 = s[i + step], w2 = s[i + 2 * step], w3 = s[i + 3 * step];
      d[i] = w0;
      d[i + step] = w1;
      d[i + 2 * step] = w2;
      d[i + 3 * step] = w3;
    }
    for (; i < words; i += step) d[i] = s[i];
  } else {
    const int row_words = static_cast<int>(a.rows_bytes / 16);
    const int64_t words = static_cast<int64_t>(a.kv_heads) * a.page_tokens * row_words;
    for (int64_t i = static_cast<int64_t>(piece) * kThreads + threadIdx.x; i < words;
         i += static_cast<int64_t>(kThreads) * a.pieces) {
      const int64_t row = i / row_words;
      const int64_t at = (row / a.page_tokens) * a.head[which] + (row % a.page_tokens) * a.tok[which] +
                         (i - row * row_words) * 16;
      *reinterpret_cast<u32x4*>(dst + at) = *reinterpret_cast<const u32x4*>(src + at);
    }
  }
}

// Jobs are (pair, layer, k or v, piece), piece fastest; a workgroup walks over
// them by the grid's size. `count` is on the device where the host does not
// know it.
__device__ __forceinline__ void copy_pairs(const PageArgs& a, const int32_t* src, const int32_t* dst,
                                           int64_t n, int64_t block, int64_t blocks) {
  const int64_t per = static_cast<int64_t>(a.layers) * 2 * a.pieces;
  for (int64_t job = block; job < n * per; job += blocks) {
    const int64_t pair = job / per;
    const int rest = static_cast<int>(job - pair * per);
    const int from = src[pair], to = dst[pair];
    if (static_cast<uint32_t>(from) >= static_cast<uint32_t>(a.pages) ||
        static_cast<uint32_t>(to) >= static_cast<uint32_t>(a.pages) || from == to)
      continue;
    copy_page(a, (rest / a.pieces) % 2, rest / a.pieces / 2, rest % a.pieces, from, to);
  }
}

__global__ __launch_bounds__(kThreads) void copy_kernel(PageArgs a, const int32_t* src,
                                                        const int32_t* dst, int64_t n) {
  copy_pairs(a, src, dst, n, blockIdx.x, gridDim.x);
}

__global__ __launch_bounds__(kThreads) void free_kernel(int32_t* refs, int pages, int32_t* tables,
                                                        int slots, int width, int64_t stride,
                                                        int32_t* lens, const int32_t* rows) {
  const int row = rows[blockIdx.x];
  if (row < 0 || row >= slots) return;
  for (int i = threadIdx.x; i < width; i += kThreads) {
    // The exchange hands an entry to one of two workgroups with the same row.
    const int page = atomicExch(tables + row * stride + i, -1);
    if (page >= 0 && page < pages) atomicSub(refs + page, 1);
  }
  if (threadIdx.x == 0) lens[row] = 0;
}

// Exclusive sum over the workgroup's 1024 threads, and the total.
__device__ __forceinline__ int group_scan(int v, int* total) {
  __shared__ int sums[kListThreads / kWave];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  int x = v;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int u = __shfl_up(x, d, kWave);
    if (lane >= d) x += u;
  }
  if (lane == kWave - 1) sums[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kListThreads / kWave; ++i) {
    const int s = sums[i];
    before += i < wave ? s : 0;
    all += s;
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

struct TableArgs {
  int32_t* refs;
  int32_t* tables;
  int32_t* lens;
  const int32_t* parents;
  const int32_t* children;
  int32_t* status;
  int64_t stride;
  int slots, width, n, pages, page;
  // Workspace.
  int32_t* claim;  // [slots]: the first fork that names this child
  int32_t* src;    // [n or pages]: pages to copy, -1 for none
  int32_t* dst;
  int32_t* len;    // [n]: the parent's length before the call; -1: the fork is refused
  int32_t* map;    // [pages]
  int32_t* count;
};

// Forks, first launch, for up to 1024 of up to kFewSlots rows: a thread keeps
// its fork in registers, claims and fresh pages stay in LDS, so the launch is
// four trips to memory (8 us; 10 by the lists in memory).
constexpr int kFewSlots = 4096;
__global__ __launch_bounds__(kListThreads) void fork_few_kernel(TableArgs a) {
  const int tid = threadIdx.x;
  __shared__ int claim[kFewSlots], parent[kListThreads], pages_of[kListThreads], bad[kListThreads];
  __shared__ int fresh[kListThreads];
  const int c = tid < a.n ? a.children[tid] : -1, p = tid < a.n ? a.parents[tid] : -1;
  int ref[kRun];
#pragma unroll
  for (int k = 0; k < kRun; ++k) ref[k] = tid * kRun + k < a.pages ? a.refs[tid * kRun + k] : 1;
  for (int i = tid; i < a.slots; i += kListThreads) claim[i] = a.n;
  pages_of[tid] = 0;
  bad[tid] = 0;
  __syncthreads();
  if (c >= 0 && c < a.slots) atomicMin(claim + c, tid);
  __syncthreads();
  int len = -1;
  if (c >= 0 && c < a.slots && p >= 0 && p < a.slots && claim[c] == tid) {
    const int own = a.lens[c], of_parent = a.lens[p];
    if (own == 0 && (static_cast<int64_t>(of_parent) + a.page - 1) / a.page <= a.width) len = of_parent;
  }
  if (len > 0) {
    parent[tid] = p;
    pages_of[tid] = static_cast<int>((static_cast<int64_t>(len) + a.page - 1) / a.page);
  }
  __syncthreads();
  // All the parents' pages, entry by entry.
  const int64_t entries = static_cast<int64_t>(a.n) * a.width;
#pragma unroll 4
  for (int64_t k = tid; k < entries; k += kListThreads) {
    const int f = static_cast<int>(k / a.width), e = static_cast<int>(k - static_cast<int64_t>(f) * a.width);
    if (e < pages_of[f] &&
        static_cast<uint32_t>(a.tables[parent[f] * a.stride + e]) >= static_cast<uint32_t>(a.pages))
      bad[f] = 1;
  }
  __syncthreads();
  if (bad[tid]) len = -1;
  const int part = len > 0 && len % a.page > 0;
  int need;
  const int mine = group_scan(part, &need);
  // The first `need` free pages, ascending, by number.
  int found = 0;
  for (int64_t p0 = 0; p0 < a.pages && found < need; p0 += kListThreads * kRun) {
    const int64_t q = p0 + tid * kRun;
    if (p0) {
#pragma unroll
      for (int k = 0; k < kRun; ++k) ref[k] = q + k < a.pages ? a.refs[q + k] : 1;
    }
    int free = 0, total;
#pragma unroll
    for (int k = 0; k < kRun; ++k) free += ref[k] == 0;
    int at = found + group_scan(free, &total);
#pragma unroll
    for (int k = 0; k < kRun; ++k)
      if (ref[k] == 0) {
        if (at < need) fresh[at] = static_cast<int>(q + k);
        ++at;
      }
    found += total;
  }
  __syncthreads();
  int from = -1, to = -1;
  if (part) {
    if (mine < found) {
      to = fresh[mine];
      from = a.tables[p * a.stride + len / a.page];
      a.refs[to] = 1;
    } else {
      len = -1;
    }
  }
  if (tid < a.n) {
    a.len[tid] = len;
    a.src[tid] = from;
    a.dst[tid] = to;
  }
  int refused;
  group_scan(tid < a.n && len < 0, &refused);
  if (tid == 0) {
    a.status[0] = refused;
    a.status[1] = max(0, need - found);
  }
}

// Forks, first launch: which are sound, and a fresh page for each that needs
// one.
__global__ __launch_bounds__(kListThreads) void fork_list_kernel(TableArgs a) {
  const int tid = threadIdx.x;
  __shared__ int parent[kListThreads], pages_of[kListThreads], bad[kListThreads];
  for (int i = tid; i < a.slots; i += kListThreads) a.claim[i] = a.n;
  __syncthreads();
  for (int i = tid; i < a.n; i += kListThreads) {
    const int c = a.children[i];
    if (c >= 0 && c < a.slots) atomicMin(a.claim + c, i);
  }
  __syncthreads();
  // 1024 forks at a time: which are sound, and the number of each among those
  // that need a fresh page.
  int need = 0, refused = 0;
  for (int i0 = 0; i0 < a.n; i0 += kListThreads) {
    const int i = i0 + tid;
    int len = -1;
    pages_of[tid] = 0;
    bad[tid] = 0;
    if (i < a.n) {
      const int c = a.children[i], p = a.parents[i];
      if (c >= 0 && c < a.slots && p >= 0 && p < a.slots &&
          __hip_atomic_load(a.claim + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == i) {
        const int own = a.lens[c], of_parent = a.lens[p];
        if (own == 0 && (static_cast<int64_t>(of_parent) + a.page - 1) / a.page <= a.width) len = of_parent;
      }
      if (len > 0) {
        parent[tid] = p;
        pages_of[tid] = static_cast<int>((static_cast<int64_t>(len) + a.page - 1) / a.page);
      }
    }
    __syncthreads();
    // All the parents' pages, entry by entry.
    const int64_t entries = static_cast<int64_t>(min(kListThreads, a.n - i0)) * a.width;
#pragma unroll 4
    for (int64_t k = tid; k < entries; k += kListThreads) {
      const int f = static_cast<int>(k / a.width), e = static_cast<int>(k - static_cast<int64_t>(f) * a.width);
      if (e < pages_of[f] &&
          static_cast<uint32_t>(a.tables[parent[f] * a.stride + e]) >= static_cast<uint32_t>(a.pages))
        bad[f] = 1;
    }
    __syncthreads();
    if (bad[tid]) len = -1;
    const int part = len > 0 && len % a.page > 0;
    refused += i < a.n && len < 0;
    int total;
    const int at = need + group_scan(part, &total);
    if (i < a.n) {
      a.len[i] = len;
      a.src[i] = part ? at : -1;
    }
    need += total;
  }
  __syncthreads();
  // The first `need` free pages, ascending, into the map by number; a thread
  // takes kRun pages in a row.
  int found = 0;
  for (int64_t p0 = 0; p0 < a.pages && found < need; p0 += kListThreads * kRun) {
    const int64_t p = p0 + tid * kRun;
    int ref[kRun], mine = 0;
#pragma unroll
    for (int k = 0; k < kRun; ++k) ref[k] = p + k < a.pages ? a.refs[p + k] : 1;
#pragma unroll
    for (int k = 0; k < kRun; ++k) mine += ref[k] == 0;
    int total;
    int at = found + group_scan(mine, &total);
#pragma unroll
    for (int k = 0; k < kRun; ++k)
      if (ref[k] == 0) {
        if (at < need) a.map[at] = static_cast<int>(p + k);
        ++at;
      }
    found += total;
  }
  __syncthreads();
  for (int i = tid; i < a.n; i += kListThreads) {
    const int at = a.src[i];
    int from = -1, to = -1;
    if (at >= 0) {
      if (at < found) {
        to = a.map[at];
        from = a.tables[a.parents[i] * a.stride + a.len[i] / a.page];
        a.refs[to] = 1;
      } else {
        a.len[i] = -1;
        ++refused;
      }
    }
    a.src[i] = from;
    a.dst[i] = to;
  }
  int total;
  group_scan(refused, &total);
  if (tid == 0) {
    a.status[0] = total;
    a.status[1] = max(0, need - found);
  }
}

// Forks, second launch: workgroup i < n writes fork i's row, the others move
// pages.
__global__ __launch_bounds__(kThreads) void fork_kernel(TableArgs a, PageArgs pa) {
  if (static_cast<int>(blockIdx.x) < a.n) {
    const int i = blockIdx.x;
    const int len = a.len[i];
    if (len < 0) return;
    const int full = len / a.page, to = a.dst[i];
    const int32_t* from_row = a.tables + a.parents[i] * a.stride;
    int32_t* row = a.tables + a.children[i] * a.stride;
    for (int k = threadIdx.x; k < a.width; k += kThreads) {
      int page = -1;
      if (k < full) {
        page = from_row[k];
        atomicAdd(a.refs + page, 1);
      } else if (k == full) {
        page = to;
      }
      row[k] = page;
    }
    if (threadIdx.x == 0) a.lens[a.children[i]] = len;
    return;
  }
  copy_pairs(pa, a.src, a.dst, a.n, blockIdx.x - a.n, gridDim.x - a.n);
}

// Compaction, first launch, for up to kListThreads * kRun pages: a thread keeps
// its pages' counts in registers and finds each mover's hole in LDS. Page k *
// 1024 + t is thread t's, so that every access is a wave's neighbours (with
// eight pages in a row to a thread the stores took 13 us); a page's number
// among the holes or movers is that of its wave's 64 pages and a bit count.
__global__ __launch_bounds__(kListThreads) void compact_few_kernel(TableArgs a) {
  constexpr int kListWaves = kListThreads / kWave;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  __shared__ int hole_at[kListThreads * kRun / 2];  // no more holes below the live pages than half
  __shared__ int used_in[kListWaves], counts[kRun * kListWaves];
  int ref[kRun], used = 0;
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    const int page = k * kListThreads + tid;
    ref[k] = page < a.pages ? a.refs[page] : 0;
  }
#pragma unroll
  for (int k = 0; k < kRun; ++k) used += __popcll(__ballot(ref[k] > 0));
  if (lane == 0) used_in[wave] = used;
  __syncthreads();
  int live = 0;
#pragma unroll
  for (int i = 0; i < kListWaves; ++i) live += used_in[i];
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    const int page = k * kListThreads + tid;
    const uint64_t holes = __ballot(page < live && ref[k] <= 0), movers = __ballot(page >= live && ref[k] > 0);
    // At most 4096 of each before any page.
    if (lane == 0) counts[k * kListWaves + wave] = __popcll(holes) | (__popcll(movers) << 16);
  }
  __syncthreads();
  if (wave == 0) {
    const int x0 = counts[2 * lane], x1 = counts[2 * lane + 1];
    int x = x0 + x1;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int u = __shfl_up(x, d, kWave);
      if (lane >= d) x += u;
    }
    if (lane == kWave - 1) *a.count = x >> 16;
    counts[2 * lane] = x - x0 - x1;
    counts[2 * lane + 1] = x - x1;
  }
  __syncthreads();
  const uint64_t before = (1ull << lane) - 1;
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    const int page = k * kListThreads + tid;
    const bool hole = page < live && ref[k] <= 0;
    const uint64_t holes = __ballot(hole);
    if (hole) hole_at[(counts[k * kListWaves + wave] & 0xffff) + __popcll(holes & before)] = page;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kRun; ++k) {
    const int page = k * kListThreads + tid;
    const bool mover = page >= live && ref[k] > 0;
    const uint64_t movers = __ballot(mover);
    int to = page;
    if (mover) {
      const int at = (counts[k * kListWaves + wave] >> 16) + __popcll(movers & before);
      to = hole_at[at];
      a.src[at] = page;
      a.dst[at] = to;
      a.refs[to] = ref[k];
      a.refs[page] = 0;
    }
    if (page < a.pages) a.map[page] = to;
  }
  if (tid == 0) {
    a.status[0] = 0;
    a.status[1] = live;
  }
}

// Compaction, first launch: the pages that move, where every page goes, and
// the new reference counts.
__global__ __launch_bounds__(kListThreads) void compact_list_kernel(TableArgs a) {
  const int tid = threadIdx.x;
  // A thread takes kRun pages in a row, of every kListThreads * kRun; the first
  // such run stays in registers for the second pass.
  int first[kRun], mine = 0;
  auto load = [&](int64_t p, int(&ref)[kRun]) {
#pragma unroll
    for (int k = 0; k < kRun; ++k) ref[k] = p + k < a.pages ? a.refs[p + k] : 0;
  };
  load(tid * kRun, first);
#pragma unroll
  for (int k = 0; k < kRun; ++k) mine += first[k] > 0;
  for (int64_t p0 = kListThreads * kRun; p0 < a.pages; p0 += kListThreads * kRun) {
    int ref[kRun];
    load(p0 + tid * kRun, ref);
#pragma unroll
    for (int k = 0; k < kRun; ++k) mine += ref[k] > 0;
  }
  int live;
  group_scan(mine, &live);
  int holes = 0, movers = 0;
  for (int64_t p0 = 0; p0 < a.pages; p0 += kListThreads * kRun) {
    const int64_t p = p0 + tid * kRun;
    if (p0) load(p, first);
    // Both counts in one scan: a round has at most 8192 of each.
    int counts = 0;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const bool used = first[k] > 0;
      counts += p + k >= a.pages ? 0 : p + k < live ? !used : used << 16;
    }
    int total;
    const int at = group_scan(counts, &total);
    int hole = holes + (at & 0xffff), mover = movers + (at >> 16);
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      if (p + k >= a.pages) continue;
      const bool used = first[k] > 0;
      const int page = static_cast<int>(p + k);
      if (page < live && !used) a.dst[hole++] = page;
      if (page >= live && used) a.src[mover++] = page;
      a.map[page] = page;
    }
    holes += total & 0xffff;
    movers += total >> 16;
  }
  __syncthreads();
  for (int i = tid; i < movers; i += kListThreads) {
    const int from = a.src[i], to = a.dst[i];
    a.map[from] = to;
    a.refs[to] = a.refs[from];
    a.refs[from] = 0;
  }
  if (tid == 0) {
    *a.count = movers;
    a.status[0] = 0;
    a.status[1] = live;
  }
}

// Compaction, second launch: workgroup i < slots rewrites row i, the others
// move pages.
__global__ __launch_bounds__(kThreads) void compact_kernel(TableArgs a, PageArgs pa) {
  if (static_cast<int>(blockIdx.x) < a.slots) {
    int32_t* row = a.tables + blockIdx.x * a.stride;
    for (int k = threadIdx.x; k < a.width; k += kThreads) {
      const int page = row[k];
      if (page >= 0 && page < a.pages) row[k] = a.map[page];
    }
    return;
  }
  copy_pairs(pa, a.src, a.dst, *a.count, blockIdx.x - a.slots, gridDim.x - a.slots);
}

PageArgs page_args(const xq_kv& kv) {
  PageArgs a;
  const int eb = elem_bytes(kv.dtype);
  a.base[0] = static_cast<uint8_t*>(kv.k);
  a.base[1] = static_cast<uint8_t*>(kv.v);
  const int64_t* strides[2] = {kv.k_stride, kv.v_stride};
  a.rows_bytes = kv.dim * eb;
  a.whole = kv.kv_heads * kv.page * a.rows_bytes;
  for (int i = 0; i < 2; ++i) {
    a.layer[i] = strides[i][0] * eb;
    a.page[i] = strides[i][1] * eb;
    a.head[i] = strides[i][2] * eb;
    a.tok[i] = strides[i][3] * eb;
    const int64_t h = strides[i][2], t = strides[i][3];
    const bool by_head = (t == kv.dim || kv.page == 1) && (h == kv.page * kv.dim || kv.kv_heads == 1);
    const bool by_token = (h == kv.dim || kv.kv_heads == 1) && (t == kv.kv_heads * kv.dim || kv.page == 1);
    if (!by_head && !by_token) a.whole = 0;
  }
  a.layers = static_cast<int>(kv.layers);
  a.kv_heads = static_cast<int>(kv.kv_heads);
  a.page_tokens = static_cast<int>(kv.page);
  a.pages = static_cast<int>(kv.pages);
  // A workgroup moves at most 16 KB of a page (four 16-byte words a thread).
  const int64_t bytes = kv.kv_heads * kv.page * a.rows_bytes;
  a.pieces = static_cast<int>(std::clamp<int64_t>(bytes / (16 * 1024), 1, 64));
  return a;
}

// Workgroups for at most n page moves.
int64_t move_blocks(const PageArgs& a, int64_t n) {
  return std::clamp<int64_t>(std::min<int64_t>(n, 1 << 20) * a.layers * 2 * a.pieces, 1, 256 * 8 * 4);
}

TableArgs table_args(const xq_kv& kv, int32_t* refs, int32_t* tables, int64_t slots, int64_t width,
                     int64_t stride, int32_t* status, void* ws) {
  TableArgs a = {};
  a.refs = refs;
  a.tables = tables;
  a.status = status;
  a.stride = stride;
  a.slots = static_cast<int>(slots);
  a.width = static_cast<int>(width);
  a.pages = static_cast<int>(kv.pages);
  a.page = static_cast<int>(kv.page);
  int32_t* w = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kCounterRegion);
  a.count = w;
  w += 64;
  a.map = w;
  w += kv.pages;
  const int64_t list = std::max(kv.pages, slots);
  a.src = w;
  w += list;
  a.dst = w;
  w += list;
  a.len = w;
  w += slots;
  a.claim = w;
  return a;
}

}  // namespace

size_t cache_workspace_bytes(int64_t pages, int64_t slots) {
  return kCounterRegion + 4 * static_cast<size_t>(64 + pages + 2 * std::max(pages, slots) + 2 * slots);
}

hipError_t launch_cache_copy(const xq_kv& kv, const int32_t* src, const int32_t* dst, int64_t n,
                             hipStream_t stream) {
  const PageArgs a = page_args(kv);
  copy_kernel<<<dim3(static_cast<uint32_t>(move_blocks(a, n))), dim3(kThreads), 0, stream>>>(a, src, dst, n);
  return hipGetLastError();
}

hipError_t launch_cache_free(const xq_kv& kv, int32_t* refs, int32_t* tables, int64_t slots,
                             int64_t width, int64_t stride, int32_t* lens, const int32_t* rows,
                             int64_t n, hipStream_t stream) {
  free_kernel<<<dim3(static_cast<uint32_t>(n)), dim3(kThreads), 0, stream>>>(
      refs, static_cast<int>(kv.pages), tables, static_cast<int>(slots), static_cast<int>(width),
      stride, lens, rows);
  return hipGetLastError();
}

hipError_t launch_cache_fork(const xq_kv& kv, int32_t* refs, int32_t* tables, int64_t slots,
                             int64_t width, int64_t stride, int32_t* lens, const int32_t* parents,
                             const int32_t* children, int64_t n, int32_t* status, void* ws,
                             hipStream_t stream) {
  TableArgs t = table_args(kv, refs, tables, slots, width, stride, status, ws);
  t.lens = lens;
  t.parents = parents;
  t.children = children;
  t.n = static_cast<int>(n);
  if (n <= kListThreads && slots <= kFewSlots)
    fork_few_kernel<<<dim3(1), dim3(kListThreads), 0, stream>>>(t);
  else
    fork_list_kernel<<<dim3(1), dim3(kListThreads), 0, stream>>>(t);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || n == 0) return e;
  const PageArgs a = page_args(kv);
  fork_kernel<<<dim3(static_cast<uint32_t>(n + move_blocks(a, n))), dim3(kThreads), 0, stream>>>(t, a);
  return hipGetLastError();
}

hipError_t launch_cache_compact(const xq_kv& kv, int32_t* refs, int32_t* tables, int64_t slots,
                                int64_t width, int64_t stride, int32_t* status, void* ws,
                                hipStream_t stream) {
  const TableArgs t = table_args(kv, refs, tables, slots, width, stride, status, ws);
  if (kv.pages <= kListThreads * kRun)
    compact_few_kernel<<<dim3(1), dim3(kListThreads), 0, stream>>>(t);
  else
    compact_list_kernel<<<dim3(1), dim3(kListThreads), 0, stream>>>(t);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const PageArgs a = page_args(kv);
  // At most half the pages move.
  compact_kernel<<<dim3(static_cast<uint32_t>(slots + move_blocks(a, kv.pages / 2 + 1))), dim3(kThreads), 0,
                   stream>>>(t, a);
  return hipGetLastError();
}

}  // namespace xq
