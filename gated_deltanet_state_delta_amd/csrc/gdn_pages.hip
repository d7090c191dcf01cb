// gdn_pages.hip -- the pages of a cache: contents copied between pages, and
// page tables grown, forked, freed and compacted on the device.
//
// A page is free when refs[page] == 0.  Pages are always taken lowest first,
// in row order, so every result is determined by the inputs; counts are
// changed with integer atomics only, whose order does not matter.  Nothing is
// read on the host: sizes fix the launches, and the lists that a call emits
// are padded with -1.
//
// The calls are launch-bound at serving sizes (a few MB of tables and
// counts), so launches are few: extend takes two, compact three, fork four.
// One pass over the counts leaves each tile's number of free pages and their
// bits; the workgroup of a row then finds the pages of its ranks by scanning
// the tiles' numbers and the bits of the tiles that hold them.  No workgroup
// waits for another inside a launch.
#include "gdn_device.hpp"
#include "gdn_paged.hpp"

namespace gdn {

// ------------------------------------------------------------------- copy --

// 16 bytes at any alignment.
typedef u32x4 u32x4_any __attribute__((aligned(1)));

constexpr int kCopyChunk = 16384;  // bytes of a page that one workgroup copies at a time

// HBM-bound for large pages: 256 slots of 2 MiB take 188 us (5.7 TB/s read
// and written; 205 us with ordinary loads and stores, which leave the copy in
// the caches, and 206 with chunks of 128 KiB).  Pieces of 16 bytes, four loads in
// flight per thread; the last bytes of a page one by one.  Workgroups step
// over (pair, chunk) items, so a list that is mostly -1 costs its reading only.
__global__ void __launch_bounds__(256) pages_copy_kernel(char* pool, int64_t page_bytes, int64_t stride, int n_pages,
                                                         const int32_t* src, const int32_t* dst, int64_t items,
                                                         uint32_t chunks) {
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t pair = chunks == 1 ? it : it / chunks;
    const int s = src[pair], d = dst[pair];
    if (s < 0 || s >= n_pages || d < 0 || d >= n_pages || s == d) continue;
    const int64_t at = (it - pair * chunks) * kCopyChunk;
    const int bytes = (int)min((int64_t)kCopyChunk, page_bytes - at), vec = bytes / 16;
    const u32x4_any* from = reinterpret_cast<const u32x4_any*>(pool + s * stride + at);
    u32x4_any* to = reinterpret_cast<u32x4_any*>(pool + d * stride + at);
    int i = threadIdx.x;
    for (; i + 768 < vec; i += 1024) {
      u32x4 t[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) t[k] = __builtin_nontemporal_load(from + i + 256 * k);
#pragma unroll
      for (int k = 0; k < 4; ++k) __builtin_nontemporal_store(t[k], to + i + 256 * k);
    }
    for (; i < vec; i += 256) __builtin_nontemporal_store(__builtin_nontemporal_load(from + i), to + i);
    const int rest = vec * 16 + threadIdx.x;
    if (rest < bytes) ((char*)to)[rest] = ((const char*)from)[rest];
  }
}

hipError_t launch_pages_copy(void* pool, int64_t page_bytes, int64_t stride, int n_pages, const int32_t* src,
                             const int32_t* dst, int64_t n, hipStream_t stream) {
  const int64_t chunks = (page_bytes + kCopyChunk - 1) / kCopyChunk, items = n * chunks;
  const dim3 grid((unsigned)(items < 16384 ? items : 16384));
  hipLaunchKernelGGL(pages_copy_kernel, grid, dim3(256), 0, stream, (char*)pool, page_bytes, stride, n_pages, src, dst,
                     items, (uint32_t)chunks);
  return hipGetLastError();
}

// ----------------------------------------------------------- tile ranking --

constexpr int kTile = 1024;  // pages of one workgroup, 4 a thread

struct PagesParams {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* refs;
  int32_t* table_out;
  int32_t* lens_out;
  int32_t* refs_out;
  int64_t table_stride, table_out_stride;
  int rows, max_pages, n_pages, page_size, tiles;
  // workspace: per tile, ranked pages, per row and per page scratch
  int32_t* tile_n;
  uint64_t* bits;  // free pages, 16 words a tile
  int32_t* list;
  int32_t* row_a;
  int32_t* row_b;
  int32_t* page_a;
  int32_t* page_b;
  int32_t* page_c;
  int32_t* total;
};

// Sum over the workgroup's 256 threads, in every thread.
__device__ __forceinline__ int block_sum(int v, int* lds) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return lds[0] + lds[1] + lds[2] + lds[3];
}
// Sum of the values of the threads before this one; `all` gets the whole sum.
__device__ __forceinline__ int block_before(int v, int* lds, int& all) {
  int s = v;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(s, o);
    if (lane >= o) s += t;
  }
  __syncthreads();
  if (lane == 63) lds[w] = s;
  __syncthreads();
  int base = 0;
  for (int i = 0; i < w; ++i) base += lds[i];
  all = lds[0] + lds[1] + lds[2] + lds[3];
  return base + s - v;
}

__device__ __forceinline__ int row_len(const PagesParams& p, const int32_t* lens, int r) {
  const int cap = p.max_pages * p.page_size;
  return min(max(lens[r], 0), cap);
}
__device__ __forceinline__ int pages_of(const PagesParams& p, int len) { return (int)(((int64_t)len + p.page_size - 1) / p.page_size); }
__device__ __forceinline__ bool is_page(const PagesParams& p, int e) { return e >= 0 && e < p.n_pages; }

// refs -> refs_out if `copy`, and how many pages of this workgroup's tile are
// free (LIVE: in use), with their bits.
template <bool LIVE>
__device__ __forceinline__ void count_tile(const PagesParams& p, const int32_t* refs, bool copy, int* lds) {
  int n = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t i = (int64_t)blockIdx.x * kTile + k * 256 + threadIdx.x;
    bool hit = false;
    if (i < p.n_pages) {
      const int v = refs[i];
      hit = LIVE ? v > 0 : v == 0;
      if (copy) p.refs_out[i] = v;
    }
    const uint64_t bits = __ballot(hit);
    if (!LIVE && (threadIdx.x & 63) == 0) p.bits[(int64_t)blockIdx.x * 16 + k * 4 + (threadIdx.x >> 6)] = bits;
    n += hit;
  }
  n = block_sum(n, lds);
  if (threadIdx.x == 0) p.tile_n[blockIdx.x] = n;
}
// Sums of tile_n before this tile, and of all.
__device__ __forceinline__ int tiles_before(const PagesParams& p, int tile, int* lds, int& all) {
  int a = 0, t = 0;
  for (int i = threadIdx.x; i < p.tiles; i += 256) {
    const int v = p.tile_n[i];
    t += v;
    if (i < tile) a += v;
  }
  all = block_sum(t, lds);
  return block_sum(a, lds);
}

// Calls use(rank, page) once for each free page whose rank lies in [start,
// end), in any thread, from the counts and bits that count_tile left.  The
// whole workgroup calls it; returns the number of free pages up to the last
// tile that it looked at (all of them where that is at most start).
struct TileList { int n[256], before[256]; };
template <typename F>
__device__ __forceinline__ int free_pages(const PagesParams& p, int start, int end, int* lds, TileList& found, F use) {
  int base = 0;
  for (int t0 = 0; t0 < p.tiles && base < end; t0 += 256) {
    const int t = t0 + threadIdx.x, v = t < p.tiles ? p.tile_n[t] : 0;
    int all, count;
    const int before = base + block_before(v, lds, all);
    const bool holds = v > 0 && before < end && before + v > start;
    const int at = block_before(holds, lds, count);
    if (holds) {
      found.n[at] = t;
      found.before[at] = before;
    }
    __syncthreads();
    for (int i = 0; i < count; ++i) {
      const int tile = found.n[i];
      const uint32_t four = (uint32_t)(p.bits[(int64_t)tile * 16 + (threadIdx.x >> 4)] >> (4 * (threadIdx.x & 15))) & 15u;
      int unused;
      int rank = found.before[i] + block_before(__popc(four), lds, unused);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if ((four >> k) & 1) {
          if (rank >= start && rank < end) use(rank, tile * kTile + (int)threadIdx.x * 4 + k);
          ++rank;
        }
    }
    __syncthreads();
    base += all;
  }
  return base;
}

// ----------------------------------------------------------------- extend --

// Tiles count their free pages; the last workgroup sums the rows' needs in
// order: row_a, the pages that the rows before need (at most n_pages + 1), and
// row_b, the row's own, -1 where it would outgrow its table.
__global__ void __launch_bounds__(256) extend_count_kernel(PagesParams p, const int32_t* add) {
  __shared__ int lds[4];
  if ((int)blockIdx.x < p.tiles) return count_tile<false>(p, p.refs, p.refs_out != p.refs, lds);
  int64_t before = 0;
  for (int r0 = 0; r0 < p.rows; r0 += 1024) {  // four neighbouring rows a thread
    const int r = r0 + (int)threadIdx.x * 4;
    int need[4], from[4], mine = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      need[k] = -1;
      if (r + k < p.rows) {
        const int len = row_len(p, p.lens, r + k);
        const int64_t grown = (int64_t)len + max(add[r + k], 0);
        if (grown <= (int64_t)p.max_pages * p.page_size) need[k] = pages_of(p, (int)grown) - pages_of(p, len);
      }
      // a sum past the pages' number counts as n_pages + 1 (n_pages is at most
      // 2^22), so that the workgroup's sum stays below 2^31
      from[k] = mine;
      mine = min(mine + min(max(need[k], 0), p.n_pages + 1), p.n_pages + 1);
    }
    int all;
    const int64_t at = before + block_before(mine, lds, all);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (r + k < p.rows) {
        p.row_a[r + k] = (int)min(at + from[k], (int64_t)p.n_pages + 1);
        p.row_b[r + k] = need[k];
      }
    before = min(before + all, (int64_t)p.n_pages + 1);
  }
}

__global__ void __launch_bounds__(256) extend_assign_kernel(PagesParams p, const int32_t* add, int32_t* ok_out) {
  __shared__ int lds[4];
  __shared__ TileList found;
  const int r = blockIdx.x, start = p.row_a[r], need = p.row_b[r];
  const int32_t* from = p.table + r * p.table_stride;
  int32_t* to = p.table_out + r * p.table_out_stride;
  const int len = row_len(p, p.lens, r), have = pages_of(p, len);
  bool ok = need == 0;
  if (need > 0) {
    int n_free;
    tiles_before(p, 0, lds, n_free);
    ok = start <= n_free - need;  // (start is at most n_pages + 1)
  }
  const int n = ok ? need : 0;
  if (to != from)
    for (int i = threadIdx.x; i < p.max_pages; i += 256)
      if (i < have || i >= have + n) to[i] = from[i];
  if (n > 0)
    free_pages(p, start, start + n, lds, found, [&](int rank, int page) {
      to[have + rank - start] = page;
      p.refs_out[page] = 1;
    });
  __syncthreads();  // every thread has read the row's length
  if (threadIdx.x == 0) {
    ok_out[r] = ok;
    p.lens_out[r] = ok ? len + max(add[r], 0) : len;
  }
}

// ------------------------------------------------------------------- fork --

__global__ void __launch_bounds__(256) fork_init_kernel(PagesParams p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.n_pages) return;
  if (p.refs_out != p.refs) p.refs_out[i] = p.refs[i];
  p.page_a[i] = 0x7fffffff;  // lowest row that holds the page as its part-filled last one
  p.page_b[i] = 0;           // how many such rows
}

__global__ void __launch_bounds__(256) fork_rows_kernel(PagesParams p, const int32_t* parent) {
  const int r = blockIdx.x, from = parent[r];
  const bool has = from >= 0 && from < p.rows;
  const int len = has ? row_len(p, p.lens, from) : 0, used = pages_of(p, len);
  const int32_t* src = p.table + (has ? from : 0) * p.table_stride;
  const int32_t* old = p.table + r * p.table_stride;
  int32_t* to = p.table_out + r * p.table_out_stride;
  const int was = pages_of(p, row_len(p, p.lens, r));
  for (int i = threadIdx.x; i < p.max_pages; i += 256) {
    const int v = i < used ? src[i] : -1;
    to[i] = v;
    // An entry that stays changes no count: a kept row's, and the prompt that
    // forked rows share, whose pages would draw many atomics to one address.
    const int had = i < was ? old[i] : -1;
    if (had == v) continue;
    if (is_page(p, v)) atomicAdd(&p.refs_out[v], 1);
    if (is_page(p, had)) atomicSub(&p.refs_out[had], 1);
  }
  if (threadIdx.x == 0) {
    p.lens_out[r] = len;
    if (len % p.page_size != 0) {
      const int last = src[len / p.page_size];
      if (is_page(p, last)) {
        atomicMin(&p.page_a[last], r);
        atomicAdd(&p.page_b[last], 1);
      }
    }
  }
}

// Tiles count their free pages; the last workgroup ranks the rows that need
// a copy of their part-filled page.
__global__ void __launch_bounds__(256) fork_count_kernel(PagesParams p) {
  __shared__ int lds[4];
  if ((int)blockIdx.x < p.tiles) return count_tile<false>(p, p.refs_out, false, lds);
  int before = 0;
  for (int r0 = 0; r0 < p.rows; r0 += 256) {
    const int r = r0 + threadIdx.x;
    bool copies = false;
    if (r < p.rows) {
      const int len = p.lens_out[r];
      if (len % p.page_size != 0) {
        const int last = p.table_out[r * p.table_out_stride + len / p.page_size];
        copies = is_page(p, last) && !(p.page_a[last] == r && p.page_b[last] == p.refs_out[last]);
      }
    }
    int all;
    const int at = block_before(copies, lds, all);
    if (r < p.rows) p.row_a[r] = copies ? before + at : -1;
    before += all;
  }
}

__global__ void __launch_bounds__(256) fork_assign_kernel(PagesParams p, int32_t* src, int32_t* dst) {
  __shared__ int lds[4], fresh;
  __shared__ TileList found;
  const int r = blockIdx.x, rank = p.row_a[r];
  int32_t* to = p.table_out + r * p.table_out_stride;
  if (rank < 0) {
    if (threadIdx.x == 0) src[r] = dst[r] = -1;
    return;
  }
  if (threadIdx.x == 0) fresh = -1;
  free_pages(p, rank, rank + 1, lds, found, [&](int, int page) { fresh = page; });
  __syncthreads();
  const int d = fresh;
  if (d < 0) {  // no page left: the row ends empty
    for (int i = threadIdx.x; i < p.max_pages; i += 256) {
      if (is_page(p, to[i])) atomicSub(&p.refs_out[to[i]], 1);
      to[i] = -1;
    }
  }
  if (threadIdx.x == 0) {
    int s = -1;
    if (d < 0) {
      p.lens_out[r] = 0;
    } else {
      int32_t* e = to + p.lens_out[r] / p.page_size;
      s = *e;
      *e = d;
      atomicSub(&p.refs_out[s], 1);
      p.refs_out[d] = 1;
    }
    src[r] = s;
    dst[r] = d;
  }
}

// ------------------------------------------------------------------- free --

__global__ void __launch_bounds__(256) refs_copy_kernel(PagesParams p) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < p.n_pages) p.refs_out[i] = p.refs[i];
}

__global__ void __launch_bounds__(256) free_rows_kernel(PagesParams p, const uint8_t* mask) {
  const int r = blockIdx.x;
  const bool out = mask[r] != 0;
  const int len = row_len(p, p.lens, r), used = pages_of(p, len);
  const int32_t* from = p.table + r * p.table_stride;
  int32_t* to = p.table_out + r * p.table_out_stride;
  for (int i = threadIdx.x; i < p.max_pages; i += 256) {
    const int v = from[i];
    if (out && i < used && is_page(p, v)) atomicSub(&p.refs_out[v], 1);
    to[i] = out ? -1 : v;
  }
  __syncthreads();  // every thread has read the row's length
  if (threadIdx.x == 0) p.lens_out[r] = out ? 0 : len;
}

// ---------------------------------------------------------------- compact --

__global__ void __launch_bounds__(256) compact_count_kernel(PagesParams p) {
  __shared__ int lds[4];
  count_tile<true>(p, p.refs, false, lds);
}

// With n_live pages in use: list[i] = the i-th free page below n_live;
// page_a[p] = i for the i-th used page at or above it (-1: not used), with
// page_b[i] = that page and page_c[i] = its count.
__global__ void __launch_bounds__(256) compact_rank_kernel(PagesParams p) {
  __shared__ int lds[4];
  int n_live;
  int base = tiles_before(p, blockIdx.x, lds, n_live);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.total = n_live;
  // used pages below n_live: whole tiles, then the tile that n_live falls into
  const int edge = n_live / kTile;
  int unused_all;
  int front = tiles_before(p, edge, lds, unused_all);
  if (edge < p.tiles) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = (int64_t)edge * kTile + k * 256 + threadIdx.x;
      if (i < n_live) n += p.refs[i] > 0;
    }
    front += block_sum(n, lds);
  }
  const int i0 = blockIdx.x * kTile + threadIdx.x * 4;  // four neighbouring pages a thread
  int v[4], mine = 0, unused;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = i0 + k < p.n_pages ? p.refs[i0 + k] : 0;
    mine += v[k] > 0;
  }
  int rank = base + block_before(mine, lds, unused);  // used pages before page i
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = i0 + k;
    if (i < p.n_pages) {
      if (i < n_live) {
        if (v[k] <= 0) p.list[i - rank] = i;
      } else {
        p.page_a[i] = v[k] > 0 ? rank - front : -1;
        if (v[k] > 0) {
          p.page_b[rank - front] = i;
          p.page_c[rank - front] = v[k];
        }
      }
    }
    rank += v[k] > 0;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.total[1] = n_live - front;  // pages that move
}

// The first rows workgroups rewrite the table, the others counts and moves.
__global__ void __launch_bounds__(256) compact_apply_kernel(PagesParams p, int32_t* src, int32_t* dst, int32_t* n_live_out) {
  const int n_live = p.total[0], moves = p.total[1];
  if ((int)blockIdx.x < p.rows) {
    const int r = blockIdx.x;
    const int32_t* from = p.table + r * p.table_stride;
    int32_t* to = p.table_out + r * p.table_out_stride;
    for (int i = threadIdx.x; i < p.max_pages; i += 256) {
      int v = from[i];
      if (v >= n_live && v < p.n_pages) {
        const int at = p.page_a[v];
        if (at >= 0) v = p.list[at];
      }
      to[i] = v;
    }
    return;
  }
  const int64_t i = (int64_t)(blockIdx.x - p.rows) * 256 + threadIdx.x;
  if (i >= p.n_pages) return;
  if (i >= n_live) p.refs_out[i] = 0;
  else if (p.refs_out != p.refs && p.refs[i] > 0) p.refs_out[i] = p.refs[i];
  if (i < moves) p.refs_out[p.list[i]] = p.page_c[i];
  if (i < p.n_pages / 2) {
    src[i] = i < moves ? p.page_b[i] : -1;
    dst[i] = i < moves ? p.list[i] : -1;
  }
  if (i == 0) *n_live_out = n_live;
}

// ----------------------------------------------------------------- launch --

// Workspace, in int32 words: [total, padded to 64][bits, 32 a tile][tile
// counts][list, page_a, page_b, page_c: n_pages each][row_a, row_b: rows each].
size_t pages_workspace_bytes(int64_t rows, int64_t n_pages) {
  const int64_t tiles = (n_pages + kTile - 1) / kTile;
  return (size_t)(64 + 33 * tiles + 4 * n_pages + 2 * rows) * sizeof(int32_t);
}

static PagesParams pages_params(const gdn_pages_args& a) {
  PagesParams p;
  p.table = a.page_table;
  p.lens = a.lens;
  p.refs = a.refs;
  p.table_out = a.page_table_out;
  p.lens_out = a.lens_out;
  p.refs_out = a.refs_out;
  p.table_stride = a.page_table_stride;
  p.table_out_stride = a.page_table_out_stride;
  p.rows = a.rows;
  p.max_pages = a.max_pages;
  p.n_pages = a.n_pages;
  p.page_size = a.page_size;
  p.tiles = (a.n_pages + kTile - 1) / kTile;
  p.total = (int32_t*)a.workspace;
  p.bits = (uint64_t*)(p.total + 64);
  p.tile_n = p.total + 64 + 32 * p.tiles;
  p.list = p.tile_n + p.tiles;
  p.page_a = p.list + a.n_pages;
  p.page_b = p.page_a + a.n_pages;
  p.page_c = p.page_b + a.n_pages;
  p.row_a = p.page_c + a.n_pages;
  p.row_b = p.row_a + a.rows;
  return p;
}

hipError_t launch_pages_extend(const gdn_pages_args& a, const int32_t* add, int32_t* ok, hipStream_t stream) {
  const PagesParams p = pages_params(a);
  hipLaunchKernelGGL(extend_count_kernel, dim3(p.tiles + 1), dim3(256), 0, stream, p, add);
  if (p.rows > 0) hipLaunchKernelGGL(extend_assign_kernel, dim3(p.rows), dim3(256), 0, stream, p, add, ok);
  return hipGetLastError();
}

hipError_t launch_pages_fork(const gdn_pages_args& a, const int32_t* parent, int32_t* src, int32_t* dst, hipStream_t stream) {
  const PagesParams p = pages_params(a);
  hipLaunchKernelGGL(fork_init_kernel, dim3((p.n_pages + 255) / 256), dim3(256), 0, stream, p);
  if (p.rows == 0) return hipGetLastError();
  hipLaunchKernelGGL(fork_rows_kernel, dim3(p.rows), dim3(256), 0, stream, p, parent);
  hipLaunchKernelGGL(fork_count_kernel, dim3(p.tiles + 1), dim3(256), 0, stream, p);
  hipLaunchKernelGGL(fork_assign_kernel, dim3(p.rows), dim3(256), 0, stream, p, src, dst);
  return hipGetLastError();
}

hipError_t launch_pages_free(const gdn_pages_args& a, const uint8_t* mask, hipStream_t stream) {
  const PagesParams p = pages_params(a);
  if (p.refs_out != p.refs)
    hipLaunchKernelGGL(refs_copy_kernel, dim3((p.n_pages + 255) / 256), dim3(256), 0, stream, p);
  if (p.rows > 0) hipLaunchKernelGGL(free_rows_kernel, dim3(p.rows), dim3(256), 0, stream, p, mask);
  return hipGetLastError();
}

hipError_t launch_pages_compact(const gdn_pages_args& a, int32_t* src, int32_t* dst, int32_t* n_live, hipStream_t stream) {
  const PagesParams p = pages_params(a);
  hipLaunchKernelGGL(compact_count_kernel, dim3(p.tiles), dim3(256), 0, stream, p);
  hipLaunchKernelGGL(compact_rank_kernel, dim3(p.tiles), dim3(256), 0, stream, p);
  hipLaunchKernelGGL(compact_apply_kernel, dim3(p.rows + (p.n_pages + 255) / 256), dim3(256), 0, stream, p, src, dst, n_live);
  return hipGetLastError();
}

}  // namespace gdn
