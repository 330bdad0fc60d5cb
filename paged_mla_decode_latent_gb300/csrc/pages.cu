// pages.cu -- the pages of a cache: sequences that grow, shrink and end
// (resize), go on from one another (fork), and live pages moved together
// (compact), all decided on the GPU.
//
// A book of pages is refs[p], how many rows hold page p (0: free), a block
// table and its lengths.  Pages are handed out lowest first, which makes the
// result a matter of the arguments alone: the k-th page asked for is the k-th
// zero of refs.  Finding those is a prefix sum over refs, done in two passes: a
// count for each chunk of 4096 pages, then, with the counts before a chunk
// added up by its CTA, the ranks inside it.  Counts change by integer atomics,
// whose order does not show.
//
// A call is a chain of steps, each of which needs all of the one before.  Where
// the book is small a cluster of eight CTAs takes the steps in one launch, with the
// cluster's barrier between them; else each step is a kernel, launched while the
// one before it still runs and waiting for it (programmatic dependent launch).
// What a call wrote is visible behind the dependency wait of the kernel after it, where
// the inserts and the device planner read it; the decode kernels read the lengths before
// they wait, but their calls queue a memset first, which no launch overlaps.  A call's last
// kernel triggers no early start on top of that.
// Moving rows is a kernel of its own, over the whole GPU, unless they are few.
//
// refs and the tables are small (4 bytes a page or entry), so resize is bound by
// the latency of its three kernels, fork and compact by those and by the rows
// that they move, 16 bytes a thread and access, four in flight a thread.

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "../../include/mla_decode.h"
#include "ptx.cuh"

namespace {

constexpr int kThreads = 512;
constexpr int kPer = 8;                   // pages a thread looks at in a chunk
constexpr int kChunk = kThreads * kPer;   // 4096
constexpr int kWarps = kThreads / 32;
constexpr int kSlice = 256;               // table entries a warp takes at a time
constexpr int kSegment = 4 * 16 * kThreads;  // bytes that a CTA moves at a time
constexpr int kMaxRows = 65535;
constexpr int kCluster = 8;
// What a cluster takes alone.  On the GPU it is no faster than the chain (resize and fork
// of 64 rows, us in a graph: 5.6 and 6.3 against 5.8 and 5.9 at 4096 pages, 6.0 and 7.5
// against 5.5 and 6.8 at 32768, 7.4 and 9.2 against 5.9 and 7.4 at 65536), but the host
// spends 4 us less on a call (8 against 12 for resize, 13 against 17 for fork).
constexpr int64_t kClusterPages = 1 << 15, kClusterEntries = 1 << 18;
// And the bytes up to which it copies fork's rows, too (8 beams, us in a graph and of the
// host: 10.1 and 10.8 against 10.6 and 13.1 by a kernel of its own at 72 KB, 12.4 and 10.8
// against 11.7 and 12.9 at 288 KB).
constexpr int64_t kClusterBytes = 1 << 17;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align256(int64_t a) { return ceil_div(a, 256) * 256; }

struct Totals {
  int32_t wanted;  // resize: pages asked for; fork: copies; both at most 2^31 - 1
  int32_t given;   // fork: copies that found a page; compact: pages to move
  int32_t live;    // compact
};

struct Book {
  int32_t* refs;
  int64_t pages;
  int32_t* status;  // or nullptr
  int page_size;
  // workspace
  Totals* totals;
  int32_t* count;  // [chunks]: free (resize, fork) or live (compact) pages
  int32_t *row_a, *row_b, *row_c;   // [rows]
  int32_t *page_a, *page_b, *page_c;  // [pages]
  int chunks;
};

struct Table {
  int32_t* at;
  int64_t stride;
  int width;  // entries a row has room for
  int32_t* lens;
  int rows;
};

struct Cache {
  uint8_t* at;
  int64_t layer_stride, row_bytes;
  int layers;
};

__device__ __forceinline__ void flag(const Book& k, int32_t bit) {
  if (k.status != nullptr) atomicOr(k.status, bit);
}

// A length as the table can hold it.
__device__ __forceinline__ int length(const Book& k, const Table& t, int len) {
  const int64_t most = min((int64_t)t.width * k.page_size, (int64_t)INT32_MAX);
  if (len >= 0 && len <= most) return len;
  flag(k, MLA_DEVFLAG_CTX_RANGE);
  return len < 0 ? 0 : (int)most;
}

__device__ __forceinline__ int pages_of(int len, int page_size) {
  return (int)(((uint32_t)len + (uint32_t)page_size - 1u) / (uint32_t)page_size);  // len >= 0: below 2^32
}

__device__ __forceinline__ bool known(const Book& k, int page) {
  if (page >= 0 && page < k.pages) return true;
  flag(k, MLA_DEVFLAG_BAD_PAGE);
  return false;
}

// Sum over the CTA of `v`, and of the threads before this one (exclusive).
template <class T>
__device__ T block_scan(T v, T* before) {
  __shared__ T part[kThreads / 32 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();  // part's readers of the call before
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    T w = lane < kThreads / 32 ? part[lane] : 0;
    const T own = w;
#pragma unroll
    for (int o = 1; o < kThreads / 32; o <<= 1) {
      const T u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    if (lane < kThreads / 32) part[lane] = w - own;
    if (lane == kThreads / 32 - 1) part[kThreads / 32] = w;
  }
  __syncthreads();
  *before = part[warp] + inc - v;
  return part[kThreads / 32];
}

// The counts of all chunks, and of those before `chunk`.
__device__ int chunk_sums(const Book& k, int chunk, int* before) {
  int all = 0, mine = 0, unused;
  if (k.chunks <= 32) {  // each warp for itself
    const int lane = threadIdx.x & 31, v = lane < k.chunks ? k.count[lane] : 0;
    *before = __reduce_add_sync(0xffffffffu, lane < chunk ? v : 0);
    return __reduce_add_sync(0xffffffffu, v);
  }
  for (int c = threadIdx.x; c < k.chunks; c += kThreads) {
    const int v = k.count[c];
    all += v;
    if (c < chunk) mine += v;
  }
  *before = block_scan(mine, &unused);
  return block_scan(all, &unused);
}

// The eight counts of refs from `at` on (past the end: a page that is held).
__device__ __forceinline__ void load_refs(const Book& k, int64_t at, int (&v)[kPer]) {
  if (at + kPer <= k.pages) {
    const int4 a = *reinterpret_cast<const int4*>(k.refs + at);
    const int4 b = *reinterpret_cast<const int4*>(k.refs + at + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) v[i] = at + i < k.pages ? k.refs[at + i] : INT32_MIN;
}

// One chunk's free (or live) pages.  A count below zero is a book that does not
// add up.
template <bool kLive>
__device__ void count_chunk(const Book& k, int chunk) {
  int v[kPer], n = 0, unused;
  load_refs(k, (int64_t)chunk * kChunk + threadIdx.x * kPer, v);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    n += kLive ? v[i] > 0 : v[i] == 0;
    if (v[i] < 0 && v[i] != INT32_MIN) flag(k, MLA_DEVFLAG_REFS);
  }
  const int all = block_scan(n, &unused);
  if (threadIdx.x == 0) k.count[chunk] = all;
}

// --------------------------------------------------------------- resize ---

// The pages that each row needs, and those needed before it.
__device__ void resize_needs(const Book& k, const Table& t, const int32_t* new_lens) {
  int64_t sum = 0;
  for (int b0 = 0; b0 < t.rows; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int need = 0;
    if (b < t.rows) {
      const int old = length(k, t, t.lens[b]);
      need = max(0, pages_of(length(k, t, new_lens[b]), k.page_size) - pages_of(old, k.page_size));
      k.row_b[b] = old;
    }
    // A row that 2^31 - 1 pages or more are asked for before gets none: there are fewer.
    int64_t before;
    const int64_t all = block_scan((int64_t)need, &before);
    if (b < t.rows) k.row_a[b] = (int)min(sum + before, (int64_t)INT32_MAX);
    sum += all;
  }
  if (threadIdx.x == 0) k.totals->wanted = (int)min(sum, (int64_t)INT32_MAX);
}

// A warp's slices of the rows: CTA `id` of `n`.
struct Slices {
  int64_t u, end, step;
  int lane;
  __device__ Slices(int64_t count, int id, int n)
      : u((int64_t)id * kWarps + (threadIdx.x >> 5)), end(count), step((int64_t)n * kWarps), lane(threadIdx.x & 31) {}
};

// Pages that rows give back: CTA `id` of `n`.
__device__ void resize_release(const Book& k, const Table& t, const int32_t* new_lens, int slices, int id, int n) {
  const Slices w((int64_t)t.rows * slices, id, n);
  for (int64_t u = w.u; u < w.end; u += w.step) {
    const int b = (int)(u / slices), j0 = (int)(u % slices) * kSlice;
    const int first = max(j0, pages_of(length(k, t, new_lens[b]), k.page_size));
    const int end = min(j0 + kSlice, pages_of(length(k, t, t.lens[b]), k.page_size));
    for (int j = first + w.lane; j < end; j += 32) {
      const int page = t.at[b * t.stride + j];
      if (known(k, page)) atomicSub(&k.refs[page], 1);
    }
  }
}

// What row b gets.
struct Grant {
  int old_len, len, held;  // held: the pages that it had
  bool given;
};

__device__ __forceinline__ Grant granted(const Book& k, const Table& t, const int32_t* new_lens, int b,
                                         int free_pages) {
  Grant g;
  g.old_len = k.row_b[b];
  g.held = pages_of(g.old_len, k.page_size);
  const int want = length(k, t, new_lens[b]);
  const int need = max(0, pages_of(want, k.page_size) - g.held);
  g.given = need == 0 || (int64_t)k.row_a[b] + need <= free_pages;
  g.len = g.given ? want : g.old_len;
  return g;
}

// The rows' lengths, and the slots of tokens in pages that they had: CTA `id` of `n`.
// Such a token lies in the row's last, partly filled page.  Where others hold that page
// the place is theirs too (a row that was cut back into a shared page): no slot.
__device__ void resize_rows(const Book& k, const Table& t, const int32_t* new_lens, int64_t* slots, int tokens,
                            int free_pages, int id, int n) {
  const int per = max(tokens, 1);
  for (int64_t i = (int64_t)id * kThreads + threadIdx.x; i < (int64_t)t.rows * per; i += (int64_t)n * kThreads) {
    const int b = (int)(i / per), c = (int)(i % per);
    const Grant g = granted(k, t, new_lens, b, free_pages);
    if (c == 0) {
      if (!g.given) flag(k, MLA_DEVFLAG_NO_PAGES);
      t.lens[b] = g.len;
      if (g.len > g.old_len && g.old_len % k.page_size != 0) {  // it grows in a page that it had
        const int page = t.at[b * t.stride + g.held - 1];
        if (known(k, page) && k.refs[page] > 1) flag(k, MLA_DEVFLAG_SHARED);
      }
    }
    if (tokens == 0) continue;
    const int pos = g.len - tokens + c;
    if (pos < g.old_len) {
      slots[i] = -1;
    } else if (pos / k.page_size < g.held) {
      const int page = t.at[b * t.stride + g.held - 1];
      slots[i] = known(k, page) && k.refs[page] <= 1 ? (int64_t)page * k.page_size + pos % k.page_size : -1;
    }
  }
}

// The free pages of a chunk go to the rows that asked.  `before`: those of earlier chunks.
__device__ void resize_give(const Book& k, const Table& t, const int32_t* new_lens, int64_t* slots, int tokens, int chunk,
                            int free_pages, int before) {
  // The chunk's free pages in a row first, then a page a thread: they are few, and
  // eight times the work below in every warp that holds one of them took 20 us at
  // 1.5 million pages and 256 rows, against 8.
  __shared__ uint16_t list[kChunk];
  const int wanted = k.totals->wanted;
  if (before >= wanted) return;
  int v[kPer], n = 0, at;
  const int64_t p0 = (int64_t)chunk * kChunk;
  load_refs(k, p0 + threadIdx.x * kPer, v);
#pragma unroll
  for (int i = 0; i < kPer; ++i) n += v[i] == 0;
  __syncthreads();  // list's readers of the chunk before
  const int all = min(block_scan(n, &at), wanted - before);
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (v[i] == 0) list[at++] = (uint16_t)(threadIdx.x * kPer + i);
  __syncthreads();
  for (int i = threadIdx.x; i < all; i += kThreads) {
    const int r = before + i;
    int b = 0, hi = t.rows;  // the last row that has asked for r or fewer pages before it
    while (hi - b > 1) {
      const int mid = (b + hi) / 2;
      if (k.row_a[mid] <= r) b = mid;
      else hi = mid;
    }
    const Grant g = granted(k, t, new_lens, b, free_pages);
    if (!g.given) continue;
    const int j = g.held + (r - k.row_a[b]);
    const int64_t page = p0 + list[i];
    t.at[b * t.stride + j] = (int32_t)page;
    k.refs[page] = 1;
    // the tokens asked about that this page holds
    const int64_t start = (int64_t)j * k.page_size, from = (int64_t)g.len - tokens;
    if (tokens > 0)
      for (int64_t pos = max(start, max(from, (int64_t)g.old_len)); pos < min(start + k.page_size, (int64_t)g.len); ++pos)
        slots[(int64_t)b * tokens + (pos - from)] = page * k.page_size + (pos - start);
  }
}

__global__ void __launch_bounds__(kThreads) resize_ask_kernel(Book k, Table t, const int32_t* new_lens,
                                                              int slices) {
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  if (blockIdx.x == 0) resize_needs(k, t, new_lens);
  else resize_release(k, t, new_lens, slices, blockIdx.x - 1, gridDim.x - 1);
}

__global__ void __launch_bounds__(kThreads) count_free_kernel(Book k) {
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  count_chunk<false>(k, blockIdx.x);
}

__global__ void __launch_bounds__(kThreads) resize_give_kernel(Book k, Table t, const int32_t* new_lens,
                                                               int64_t* slots, int tokens) {
  ptx::grid_dependency_wait();
  int before;
  const int chunk = min((int)blockIdx.x, k.chunks), free_pages = chunk_sums(k, chunk, &before);
  if (chunk < k.chunks) resize_give(k, t, new_lens, slots, tokens, chunk, free_pages, before);
  else resize_rows(k, t, new_lens, slots, tokens, free_pages, blockIdx.x - k.chunks, gridDim.x - k.chunks);
}

// All of it by one cluster.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    resize_kernel(Book k, Table t, const int32_t* new_lens, int slices, int64_t* slots, int tokens) {
  const int id = blockIdx.x;
  ptx::grid_dependency_wait();
  if (id == 0) resize_needs(k, t, new_lens);
  resize_release(k, t, new_lens, slices, kCluster - 1 - id, kCluster);
  ptx::cluster_sync_all();
  for (int c = id; c < k.chunks; c += kCluster) count_chunk<false>(k, c);
  ptx::cluster_sync_all();
  int before, free_pages = chunk_sums(k, id, &before);
  for (int c = id; c < k.chunks; c += kCluster) {
    if (c != id) free_pages = chunk_sums(k, c, &before);
    resize_give(k, t, new_lens, slots, tokens, c, free_pages, before);
  }
  resize_rows(k, t, new_lens, slots, tokens, free_pages, kCluster - 1 - id, kCluster);
}

// ----------------------------------------------------------------- fork ---

struct Children {
  const int32_t* parents;
  int32_t* table;
  int64_t stride;
  int32_t* lens;
  int rows;
};

// Which children need a copy of their parent's last page.
__device__ void fork_needs(const Book& k, const Table& t, const Children& c) {
  int32_t* first = k.row_a;  // a parent's first child
  for (int r = threadIdx.x; r < t.rows; r += kThreads) first[r] = INT32_MAX;
  __syncthreads();
  for (int i = threadIdx.x; i < c.rows; i += kThreads) {
    const int r = c.parents[i];
    if (r >= 0 && r < t.rows) atomicMin(&first[r], i);
    else if (r != -1) flag(k, MLA_DEVFLAG_BAD_ROW);
  }
  __syncthreads();
  int sum = 0;
  for (int i0 = 0; i0 < c.rows; i0 += kThreads) {
    const int i = i0 + threadIdx.x, r = i < c.rows ? c.parents[i] : -1;
    const int copies = r >= 0 && r < t.rows && length(k, t, t.lens[r]) % k.page_size != 0 && __ldcg(&first[r]) != i;
    int before;
    const int all = block_scan(copies, &before);
    if (copies) k.row_b[sum + before] = i;
    sum += all;
  }
  if (threadIdx.x == 0) k.totals->wanted = sum;
}

// The parents' counts, by children - 1 for whole pages, and for a partly filled
// last page by the one child that keeps it: CTA `id` of `n`.
__device__ void fork_release(const Book& k, const Table& t, const Children& c, int slices, int id, int n) {
  const Slices w((int64_t)t.rows * slices, id, n);
  for (int64_t u = w.u; u < w.end; u += w.step) {
    const int r = (int)(u / slices), j0 = (int)(u % slices) * kSlice;
    const int len = length(k, t, t.lens[r]), whole = len / k.page_size;
    const int end = min(j0 + kSlice, pages_of(len, k.page_size));
    if (j0 >= end) continue;
    int children = 0;
    for (int i = w.lane; i < c.rows; i += 32) children += c.parents[i] == r;
    children = __reduce_add_sync(0xffffffffu, children);
    if (children == 1) continue;
    for (int j = j0 + w.lane; j < end; j += 32) {
      const int page = t.at[r * t.stride + j];
      const int change = (j < whole ? children : min(children, 1)) - 1;
      if (known(k, page) && change != 0) atomicAdd(&k.refs[page], change);
    }
  }
}

// The children's rows: CTA `id` of `n`.
__device__ void fork_rows(const Book& k, const Table& t, const Children& c, int slices, int id, int n) {
  const Slices w((int64_t)c.rows * slices, id, n);
  for (int64_t u = w.u; u < w.end; u += w.step) {
    const int i = (int)(u / slices), j0 = (int)(u % slices) * kSlice, r = c.parents[i];
    const int len = r >= 0 && r < t.rows ? length(k, t, t.lens[r]) : 0;
    if (j0 == 0 && w.lane == 0) c.lens[i] = len;
    const int end = min(j0 + kSlice, pages_of(len, k.page_size));
    for (int j = j0 + w.lane; j < end; j += 32) c.table[i * c.stride + j] = t.at[r * t.stride + j];
  }
}

// The k-th free page goes to the k-th child that needs one: those of a chunk.
__device__ void fork_give(const Book& k, const Children& c, int chunk) {
  const int wanted = k.totals->wanted;
  int before;
  const int free_pages = chunk_sums(k, chunk, &before);
  if (chunk == 0) {
    if (threadIdx.x == 0) k.totals->given = min(wanted, free_pages);
    // Children that find none keep their parent's whole pages.
    for (int r = free_pages + threadIdx.x; r < wanted; r += kThreads) {
      const int i = k.row_b[r];
      c.lens[i] -= c.lens[i] % k.page_size;
      flag(k, MLA_DEVFLAG_NO_PAGES);
    }
  }
  if (before >= wanted) return;
  int v[kPer], n = 0, r;
  const int64_t p0 = (int64_t)chunk * kChunk + threadIdx.x * kPer;
  load_refs(k, p0, v);
#pragma unroll
  for (int i = 0; i < kPer; ++i) n += v[i] == 0;
  block_scan(n, &r);
  r += before;
  for (int i = 0; i < kPer; ++i) {
    if (v[i] != 0) continue;
    if (r >= wanted) break;
    const int child = k.row_b[r], j = c.lens[child] / k.page_size;
    c.table[child * c.stride + j] = (int32_t)(p0 + i);
    k.refs[p0 + i] = 1;
    k.row_c[r] = (int32_t)(p0 + i);
    ++r;
  }
}

__global__ void __launch_bounds__(kThreads) fork_ask_kernel(Book k, Table t, Children c, int slices) {
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  if (blockIdx.x == 0) fork_needs(k, t, c);
  else fork_release(k, t, c, slices, blockIdx.x - 1, gridDim.x - 1);
}

__global__ void __launch_bounds__(kThreads) fork_rows_kernel(Book k, Table t, Children c, int slices) {
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  if ((int)blockIdx.x < k.chunks) count_chunk<false>(k, blockIdx.x);
  else fork_rows(k, t, c, slices, blockIdx.x - k.chunks, gridDim.x - k.chunks);
}

__global__ void __launch_bounds__(kThreads) fork_give_kernel(Book k, Children c) {
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  fork_give(k, c, blockIdx.x);
}

// The first `bytes` bytes at `from` to `to`, by the CTA: segment `s` of them.
__device__ __forceinline__ void move_segment(uint8_t* to, const uint8_t* from, int64_t bytes, int64_t s) {
  const int64_t at = s * kSegment + threadIdx.x * 16;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (at + i * kThreads * 16 < bytes) v[i] = __ldcs(reinterpret_cast<const uint4*>(from + at + i * kThreads * 16));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (at + i * kThreads * 16 < bytes) __stcs(reinterpret_cast<uint4*>(to + at + i * kThreads * 16), v[i]);
}

// The filled rows of the pages that children get a copy of: CTA `id` of `of`.
__device__ void fork_copy(const Book& k, const Table& t, const Children& c, const Cache& cache, int id, int of) {
  const int64_t page_bytes = cache.row_bytes * k.page_size;
  const int64_t segments = (page_bytes + kSegment - 1) / kSegment;
  const int64_t units = (int64_t)__ldcg(&k.totals->given) * cache.layers * segments;
  for (int64_t u = id; u < units; u += of) {
    const int n = (int)(u / (cache.layers * segments));
    const int64_t rest = u - n * (cache.layers * segments);
    const int layer = (int)(rest / segments);
    const int child = __ldcg(&k.row_b[n]), r = c.parents[child], len = __ldcg(&c.lens[child]);
    const int from = t.at[r * t.stride + len / k.page_size], to = __ldcg(&k.row_c[n]);
    if (from < 0 || from >= k.pages) continue;  // flagged
    uint8_t* base = cache.at + layer * cache.layer_stride;
    move_segment(base + to * page_bytes, base + from * page_bytes, len % k.page_size * cache.row_bytes, rest % segments);
  }
}

__global__ void __launch_bounds__(kThreads) fork_copy_kernel(Book k, Table t, Children c, Cache cache) {
  ptx::grid_dependency_wait();
  fork_copy(k, t, c, cache, blockIdx.x, gridDim.x);
}

// The three steps by one cluster, and the copies if they are few.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    fork_kernel(Book k, Table t, Children c, Cache cache, int slices, bool copies) {
  const int id = blockIdx.x;
  ptx::grid_dependency_wait();
  if (!copies) ptx::launch_dependents();
  if (id == 0) fork_needs(k, t, c);
  fork_release(k, t, c, slices, kCluster - 1 - id, kCluster);
  fork_rows(k, t, c, slices, kCluster - 1 - id, kCluster);
  ptx::cluster_sync_all();
  for (int x = id; x < k.chunks; x += kCluster) count_chunk<false>(k, x);
  ptx::cluster_sync_all();
  for (int x = id; x < k.chunks; x += kCluster) fork_give(k, c, x);
  if (!copies) return;
  ptx::cluster_sync_all();
  fork_copy(k, t, c, cache, id, kCluster);
}

// -------------------------------------------------------------- compact ---

__global__ void __launch_bounds__(kThreads) count_live_kernel(Book k) {
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  count_chunk<true>(k, blockIdx.x);
}

// With n live pages: holes below n (page_b) and live pages from n on (page_a),
// both in order, and each of the latter's place in that order (page_c).
__device__ void compact_match(const Book& k, int32_t* map, int32_t* n_live, int chunk) {
  int before;
  const int n = chunk_sums(k, chunk, &before);
  const int64_t p0 = (int64_t)chunk * kChunk + threadIdx.x * kPer;
  int low = 0, unused;  // live pages below n
  if (chunk >= n / kChunk) {
    int at_n;
    chunk_sums(k, n / kChunk, &at_n);
    int u[kPer], c = 0;
    const int64_t q0 = (int64_t)(n / kChunk) * kChunk + threadIdx.x * kPer;
    load_refs(k, q0, u);
#pragma unroll
    for (int i = 0; i < kPer; ++i) c += u[i] > 0 && q0 + i < n;
    low = at_n + block_scan(c, &unused);
  }
  int v[kPer], c = 0, r;
  load_refs(k, p0, v);
#pragma unroll
  for (int i = 0; i < kPer; ++i) c += v[i] > 0;
  block_scan(c, &r);
  r += before;  // live pages before this one
  for (int i = 0; i < kPer; ++i) {
    const int64_t p = p0 + i;
    if (p >= k.pages) break;
    const bool live = v[i] > 0;
    if (p < n) {
      map[p] = live ? (int)p : -1;
      if (!live) k.page_b[p - r] = (int)p;
    } else {
      map[p] = -1;
      k.page_c[p] = live ? r - low : -1;
      if (live) k.page_a[r - low] = (int)p;
    }
    r += live;
  }
  if (chunk == n / kChunk || (n / kChunk == k.chunks && chunk == 0)) {
    // (n == pages at a chunk's end: every page is live, and none moves)
    if (threadIdx.x == 0) {
      k.totals->live = n;
      k.totals->given = n / kChunk == k.chunks ? 0 : n - low;
      *n_live = n;
    }
  }
}

__global__ void __launch_bounds__(kThreads) compact_match_kernel(Book k, int32_t* map, int32_t* n_live) {
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  compact_match(k, map, n_live, blockIdx.x);
}

// Both steps by one cluster.
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    compact_kernel(Book k, int32_t* map, int32_t* n_live) {
  const int id = blockIdx.x;
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  for (int x = id; x < k.chunks; x += kCluster) count_chunk<true>(k, x);
  ptx::cluster_sync_all();
  for (int x = id; x < k.chunks; x += kCluster) compact_match(k, map, n_live, x);
}

__global__ void __launch_bounds__(kThreads) compact_move_kernel(Book k, Table t, Cache cache, int32_t* map, int slices) {
  ptx::grid_dependency_wait();
  const int moves = k.totals->given, n = k.totals->live;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < moves; i += (int64_t)gridDim.x * kThreads) {
    const int from = k.page_a[i], to = k.page_b[i];
    map[from] = to;
    k.refs[to] = k.refs[from];
    k.refs[from] = 0;
  }
  const Slices w((int64_t)t.rows * slices, blockIdx.x, gridDim.x);
  for (int64_t u = w.u; u < w.end; u += w.step) {
    const int b = (int)(u / slices), j0 = (int)(u % slices) * kSlice;
    const int end = min(j0 + kSlice, pages_of(length(k, t, t.lens[b]), k.page_size));
    for (int j = j0 + w.lane; j < end; j += 32) {
      const int page = t.at[b * t.stride + j];
      if (!known(k, page)) continue;
      if (page < n) {
        if (map[page] < 0) flag(k, MLA_DEVFLAG_REFS);  // held by a row, and free
        continue;
      }
      const int place = k.page_c[page];
      if (place < 0) flag(k, MLA_DEVFLAG_REFS);
      else t.at[b * t.stride + j] = k.page_b[place];
    }
  }
  const int64_t page_bytes = cache.row_bytes * k.page_size;
  const int64_t segments = (page_bytes + kSegment - 1) / kSegment;
  const int64_t units = (int64_t)moves * cache.layers * segments;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t i = u / (cache.layers * segments), rest = u - i * (cache.layers * segments);
    uint8_t* base = cache.at + rest / segments * cache.layer_stride;
    move_segment(base + k.page_b[i] * page_bytes, base + k.page_a[i] * page_bytes, page_bytes, rest % segments);
  }
}

// ----------------------------------------------------------------- host ---

bool misaligned(const void* x, uintptr_t a) { return (reinterpret_cast<uintptr_t>(x) % a) != 0; }

int64_t carve(Book* k, char* ws, int64_t pages, int64_t rows) {
  int64_t off = 0;
  auto take = [&](auto** at, int64_t bytes) {
    if (k != nullptr) *at = reinterpret_cast<std::remove_reference_t<decltype(**at)>*>(ws + off);
    off = align256(off + bytes);
  };
  Book none;
  Book& b = k != nullptr ? *k : none;
  const int64_t chunks = ceil_div(pages, kChunk);
  take(&b.totals, sizeof(Totals));
  take(&b.count, 4 * chunks);
  take(&b.row_a, 4 * rows);
  take(&b.row_b, 4 * rows);
  take(&b.row_c, 4 * rows);
  take(&b.page_a, 4 * pages);
  take(&b.page_b, 4 * pages);
  take(&b.page_c, 4 * pages);
  return off;
}

bool sizes_fit(int64_t pages, int64_t rows) { return pages >= 1 && pages < INT32_MAX && rows >= 0 && rows <= kMaxRows; }

int make_book(Book* k, int32_t* refs, int64_t pages, int64_t rows, int page_size, int32_t* status, void* ws,
              size_t ws_bytes) {
  if (!sizes_fit(pages, rows) || page_size < 1 || page_size > 4096) return MLA_ERR_INVALID_ARG;
  if (refs == nullptr || misaligned(refs, 16) || misaligned(status, 4)) return MLA_ERR_INVALID_ARG;
  if (ws == nullptr || misaligned(ws, 256)) return MLA_ERR_WORKSPACE;
  k->refs = refs;
  k->pages = pages;
  k->status = status;
  k->page_size = page_size;
  k->chunks = (int)ceil_div(pages, kChunk);
  return carve(k, static_cast<char*>(ws), pages, rows) <= (int64_t)ws_bytes ? MLA_OK : MLA_ERR_WORKSPACE;
}

int make_table(Table* t, const int32_t* at, int64_t stride, int width, const int32_t* lens, int rows) {
  *t = Table{const_cast<int32_t*>(at), stride, width, const_cast<int32_t*>(lens), rows};
  if (rows == 0) return MLA_OK;
  if (at == nullptr || lens == nullptr || misaligned(at, 4) || misaligned(lens, 4) || width < 1 || stride < width)
    return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

int make_cache(Cache* c, void* at, int layers, int64_t layer_stride, int64_t row_bytes, int64_t pages, int page_size) {
  *c = Cache{static_cast<uint8_t*>(at), layer_stride, row_bytes, layers};
  if (at == nullptr || misaligned(at, 16) || layers < 1 || row_bytes < 16 || row_bytes % 16 != 0 ||
      row_bytes > (1 << 20))
    return MLA_ERR_INVALID_ARG;
  if (layers > 1 && (layer_stride % 16 != 0 || layer_stride / row_bytes / page_size < pages)) return MLA_ERR_INVALID_ARG;
  if (pages > INT64_MAX / 2 / row_bytes / page_size) return MLA_ERR_UNSUPPORTED;
  return MLA_OK;
}

template <class... A>
cudaError_t launch(void (*kernel)(A...), int64_t grid, void* stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// CTAs for work in pieces: all of them, up to what the GPU runs in a few rounds.
int64_t some(int64_t pieces) { return std::max<int64_t>(1, std::min<int64_t>(pieces, 152 * 8)); }

bool by_cluster(int64_t pages, int64_t rows, int64_t width) {
  return pages <= kClusterPages && rows * width <= kClusterEntries;
}

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)b_bytes && y < x + (uintptr_t)a_bytes;
}

}  // namespace

extern "C" int64_t mla_pages_workspace_bytes(int64_t num_pages, int32_t rows) {
  return sizes_fit(num_pages, rows) ? carve(nullptr, nullptr, num_pages, rows) : -1;
}

extern "C" int mla_pages_resize(int32_t* refs, int64_t num_pages, int32_t* block_table, int64_t bt_stride,
                                int32_t width, int32_t* seq_lens, const int32_t* new_lens, int32_t rows,
                                int32_t page_size, int64_t* slots, int32_t tokens, int32_t* status,
                                void* workspace, size_t workspace_bytes, void* stream) {
  Book k;
  Table t;
  int st = make_book(&k, refs, num_pages, rows, page_size, status, workspace, workspace_bytes);
  if (st == MLA_OK) st = make_table(&t, block_table, bt_stride, width, seq_lens, rows);
  if (st != MLA_OK) return st;
  if (tokens < 0 || (tokens > 0 && slots == nullptr) || misaligned(slots, 8)) return MLA_ERR_INVALID_ARG;
  if (rows == 0) return MLA_OK;
  if (new_lens == nullptr || misaligned(new_lens, 4) || overlap(new_lens, 4ll * rows, seq_lens, 4ll * rows))
    return MLA_ERR_INVALID_ARG;
  const int slices = (int)ceil_div(width, kSlice);
  if (by_cluster(num_pages, rows, width)) {
    return launch(resize_kernel, kCluster, stream, k, t, new_lens, slices, slots, (int)tokens) == cudaSuccess
               ? MLA_OK
               : MLA_ERR_CUDA;
  }
  if (launch(resize_ask_kernel, 1 + some(ceil_div((int64_t)rows * slices, kWarps)), stream, k, t, new_lens, slices) != cudaSuccess ||
      launch(count_free_kernel, k.chunks, stream, k) != cudaSuccess ||
      launch(resize_give_kernel, k.chunks + some(ceil_div((int64_t)rows * std::max(tokens, 1), kThreads)), stream, k, t,
             new_lens, slots, (int)tokens) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

extern "C" int mla_pages_fork(int32_t* refs, int64_t num_pages, const int32_t* block_table, int64_t bt_stride,
                              int32_t width, const int32_t* seq_lens, int32_t rows, const int32_t* parents,
                              int32_t* table_out, int64_t out_stride, int32_t* lens_out, int32_t out_rows,
                              int32_t page_size, void* kv_cache, int32_t layers, int64_t layer_stride,
                              int64_t row_bytes, int32_t* status, void* workspace, size_t workspace_bytes,
                              void* stream) {
  if (out_rows < 0) return MLA_ERR_INVALID_ARG;
  Book k;
  Table t;
  Cache cache;
  int st = make_book(&k, refs, num_pages, std::max(rows, out_rows), page_size, status, workspace, workspace_bytes);
  if (st == MLA_OK) st = make_table(&t, block_table, bt_stride, width, seq_lens, rows);
  if (st == MLA_OK) st = make_cache(&cache, kv_cache, layers, layer_stride, row_bytes, num_pages, page_size);
  if (st != MLA_OK) return st;
  if (rows < 1) return MLA_ERR_INVALID_ARG;
  if (out_rows > 0 && (parents == nullptr || table_out == nullptr || lens_out == nullptr || misaligned(parents, 4) ||
                       misaligned(table_out, 4) || misaligned(lens_out, 4) || out_stride < width))
    return MLA_ERR_INVALID_ARG;
  if (out_rows > 0) {  // what is written overlaps nothing else: parents are read again when rows are copied
    const int64_t table_bytes = ((rows - 1) * bt_stride + width) * 4, out_bytes = ((out_rows - 1) * out_stride + width) * 4;
    const int64_t lens_bytes = 4ll * out_rows;
    if (overlap(table_out, out_bytes, block_table, table_bytes) || overlap(table_out, out_bytes, seq_lens, 4ll * rows) ||
        overlap(table_out, out_bytes, parents, lens_bytes) || overlap(table_out, out_bytes, refs, 4 * num_pages) ||
        overlap(table_out, out_bytes, lens_out, lens_bytes) || overlap(lens_out, lens_bytes, block_table, table_bytes) ||
        overlap(lens_out, lens_bytes, seq_lens, 4ll * rows) || overlap(lens_out, lens_bytes, parents, lens_bytes) ||
        overlap(lens_out, lens_bytes, refs, 4 * num_pages))
      return MLA_ERR_INVALID_ARG;
  }
  const Children c{parents, table_out, out_stride, lens_out, out_rows};
  const int slices = (int)ceil_div(width, kSlice);
  const int64_t segments = ceil_div(row_bytes * page_size, kSegment);
  const bool cluster = by_cluster(num_pages, std::max(rows, out_rows), width);
  const bool copies = cluster && layers * row_bytes * page_size <= kClusterBytes / std::max(out_rows, 1);
  if (cluster && launch(fork_kernel, kCluster, stream, k, t, c, cache, slices, copies) != cudaSuccess) return MLA_ERR_CUDA;
  if (copies) return MLA_OK;
  if (!cluster &&
      (launch(fork_ask_kernel, 1 + some(ceil_div((int64_t)rows * slices, kWarps)), stream, k, t, c, slices) != cudaSuccess ||
       launch(fork_rows_kernel, k.chunks + some(ceil_div((int64_t)out_rows * slices, kWarps)), stream, k, t, c, slices) != cudaSuccess ||
       launch(fork_give_kernel, k.chunks, stream, k, c) != cudaSuccess))
    return MLA_ERR_CUDA;
  if (launch(fork_copy_kernel, some((int64_t)out_rows * layers * segments), stream, k, t, c, cache) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

extern "C" int mla_pages_compact(int32_t* refs, int64_t num_pages, int32_t* block_table, int64_t bt_stride,
                                 int32_t width, const int32_t* seq_lens, int32_t rows, int32_t page_size,
                                 void* kv_cache, int32_t layers, int64_t layer_stride, int64_t row_bytes,
                                 int32_t* page_map, int32_t* n_live, int32_t* status, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  Book k;
  Table t;
  Cache cache;
  int st = make_book(&k, refs, num_pages, rows, page_size, status, workspace, workspace_bytes);
  if (st == MLA_OK) st = make_table(&t, block_table, bt_stride, width, seq_lens, rows);
  if (st == MLA_OK) st = make_cache(&cache, kv_cache, layers, layer_stride, row_bytes, num_pages, page_size);
  if (st != MLA_OK) return st;
  if (page_map == nullptr || n_live == nullptr || misaligned(page_map, 4) || misaligned(n_live, 4))
    return MLA_ERR_INVALID_ARG;
  // What is written overlaps nothing else: counts that change between two reads give ranks below zero.
  const int64_t page_bytes = 4 * num_pages, table_bytes = rows > 0 ? ((rows - 1) * bt_stride + width) * 4 : 0;
  if (overlap(page_map, page_bytes, refs, page_bytes) || overlap(n_live, 4, refs, page_bytes) ||
      overlap(page_map, page_bytes, n_live, 4) || overlap(page_map, page_bytes, block_table, table_bytes) ||
      overlap(n_live, 4, block_table, table_bytes) || overlap(page_map, page_bytes, seq_lens, 4ll * rows) ||
      overlap(n_live, 4, seq_lens, 4ll * rows))
    return MLA_ERR_INVALID_ARG;
  const int slices = rows == 0 ? 1 : (int)ceil_div(width, kSlice);
  const int64_t segments = ceil_div(row_bytes * page_size, kSegment);
  const int64_t pieces = std::max(num_pages / 2 * layers * segments, ceil_div((int64_t)rows * slices, kWarps));
  const bool cluster = by_cluster(num_pages, 0, 0);
  if (cluster && launch(compact_kernel, kCluster, stream, k, page_map, n_live) != cudaSuccess) return MLA_ERR_CUDA;
  if (!cluster && (launch(count_live_kernel, k.chunks, stream, k) != cudaSuccess ||
                   launch(compact_match_kernel, k.chunks, stream, k, page_map, n_live) != cudaSuccess))
    return MLA_ERR_CUDA;
  if (launch(compact_move_kernel, some(pieces), stream, k, t, cache, page_map, slices) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}
