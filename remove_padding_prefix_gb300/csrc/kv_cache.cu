// Upkeep of a paged key-value cache: reserve, append, fork, free, compact.
//
// State (device memory, the caller's): the pool [layers, pages, 2, kv heads, page rows,
// head size] of 16-bit values (index 0 of the third axis K, 1 V), table int32 [slots,
// max_pages] of page numbers, lens int32 [slots], refs int32 [pages] (sequences that use
// a page).  A page is free where refs is 0; pages are taken lowest number first, in the
// order of the call's list, so every result is a function of the state alone: there is
// no free list whose order could depend on history, and no atomic whose order shows
// (reference counts are only added to).  What an append or a free leaves out after an error of its own
// does depend on timing: their CTAs read the error word as they start.
//
// The kernels that decide (who gets which page, what moves where) are one CTA each: they
// read refs, 4 bytes a page, twice, against 2 * kv heads * rows * head size * 2 bytes a
// page and layer for the data, and one CTA needs no grid-wide order.  Every warp owns a
// contiguous stretch of pages; counting, one scan over the 32 warps and a second walk
// with warp scans give each free page its rank without a block barrier per chunk.  The
// kernels that move rows are flat 16-byte copies over the whole grid.
//
// The lists a caller gives (slots, counts, cu_seqlens) and the state are read on the
// device; every page number and position is checked against the pool before it is used,
// so a list or a state that is wrong records a device error and never leaves the buffers.
//
// A cache of 8-bit codes has the same state: its rows of head_dim codes move as rows of head_dim / 2 16-bit values, and
// the calls that move rows move their blocks' scale bytes with them (PageScales).
#include "kv_common.cuh"

namespace rpp {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ int warp_scan_incl(int v) {
  const int lane = lane_id();
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// the four reference counts from page p on; pages past `pages` read as -1 (neither free nor live)
__device__ __forceinline__ int4 load_refs4(const int32_t* refs, int p, int pages) {
  if (p + 4 <= pages) return *reinterpret_cast<const int4*>(refs + p);
  int4 v = make_int4(-1, -1, -1, -1);
  if (p < pages) v.x = refs[p];
  if (p + 1 < pages) v.y = refs[p + 1];
  if (p + 2 < pages) v.z = refs[p + 2];
  return v;
}

// the stretch of pages of one warp: a multiple of 128 pages, so that lanes load int4
__device__ __forceinline__ int2 warp_stretch(int pages) {
  const long long per = ((static_cast<long long>(pages) + kPlanWarps * 128 - 1) / (kPlanWarps * 128)) * 128;
  const long long a = per * warp_id();
  return make_int2(static_cast<int>(a < pages ? a : pages), static_cast<int>(a + per < pages ? a + per : pages));
}

// ---------------------------------------------------------------- reserve, and the plan of a fork
// kFork == false: slot slots[i] grows by counts[i] tokens and gets the pages it lacks.
// kFork == true: slot slots[i] (empty) becomes a copy of slot from[i]; here it gets its
// length and, where from[i] ends inside a page, a page of its own for that end (the
// pages, the table row and the reference counts of the shared part follow in
// fork_copy_kernel).  All or nothing: any error leaves the state as it was.
// That the fork is on is left for fork_copy_kernel in the state itself, the error word being anybody's:
// kForkMark in the first table entry of a destination that shares pages, and `shares` times
// kForkShare on the count of its own page, one for each CTA that copies a part of it.
// Shared memory: int32 need[n + 1] (then its exclusive scan), the slot bitmap.
constexpr int kForkMark = -0x7fffffff - 1;
constexpr int kForkShare = 1 << 17;   // above every count: a page has at most kKvMaxSlots users
constexpr int kMostShares = 8192;     // kMostShares * kForkShare + 1 is an int
static_assert(kForkShare > kKvMaxSlots && static_cast<long long>(kMostShares) * kForkShare < 0x7fffffffLL, "");
template <bool kFork>
__global__ void __launch_bounds__(kPlanThreads)
    kv_reserve_kernel(KvDims d, int32_t* table, int32_t* lens, int32_t* refs,
                      const int32_t* slots, const int32_t* counts_or_from, int n, int shares,
                      int32_t* err) {
  extern __shared__ int32_t s_need[];
  uint32_t* seen = reinterpret_cast<uint32_t*>(s_need + n + 1);
  __shared__ int s_code, s_total;
  __shared__ int s_warp[kPlanWarps];
  __shared__ Gate gate;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) s_code = 0;
  const int warp = warp_id(), lane = lane_id();
  // The list and the free pages of each warp's stretch, read together with the error word.
  const int mine_i = threadIdx.x;
  const int first = mine_i < n ? slots[mine_i] : 0;
  const int first_arg = mine_i < n ? counts_or_from[mine_i] : 0;
  const int2 st = warp_stretch(d.pages);
  int mine = 0;
  for (int p = st.x + 4 * lane; p < st.y; p += 128) {
    const int4 r = load_refs4(refs, p, d.pages);
    mine += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
  }
  if (!pass(slots, n, first, d, seen, &gate, err)) return;
  // pages that each sequence needs
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int s = i == mine_i ? first : slots[i];
    const int arg = i == mine_i ? first_arg : counts_or_from[i];
    int need = 0, code = 0;
    if constexpr (kFork) {
      const int f = arg;
      if (f < 0 || f >= d.slots || ((seen[f >> 5] >> (f & 31)) & 1u)) code = RPP_DERR_SLOT;   // no slot is both
      else if (lens[s] != 0) code = RPP_DERR_SLOT;            // a fork goes to an empty slot
      else if (!len_ok(lens[f], d)) code = RPP_DERR_LENGTH;
      else need = lens[f] % d.page_size ? 1 : 0;
    } else {
      const int old = lens[s], add = arg;
      const long long grown = static_cast<long long>(old) + add;
      if (!len_ok(old, d) || add < 0 || grown > static_cast<long long>(d.max_pages) * d.page_size) code = RPP_DERR_LENGTH;
      else need = used_pages(static_cast<int>(grown), d.page_size) - used_pages(old, d.page_size);
    }
    if (code) atomicCAS(&s_code, 0, code);
    s_need[i] = need;
  }
  __syncthreads();
  if (s_code) {
    if (threadIdx.x == 0) set_device_error(err, s_code);
    return;
  }
  // exclusive scan of the needs (slots are distinct, so the sum is at most slots * max_pages)
  int carry = 0;
  for (int base = 0; base < n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    const int v = i < n ? s_need[i] : 0;
    const int incl = warp_scan_incl(v);
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      const int w = s_warp[lane];
      const int wi = warp_scan_incl(w);
      s_warp[lane] = wi - w;
      if (lane == 31) s_total = wi;
    }
    __syncthreads();
    if (i < n) s_need[i] = carry + s_warp[warp] + incl - v;
    carry += s_total;
    __syncthreads();
  }
  const int total = carry;
  if (threadIdx.x == 0) s_need[n] = total;
  // free pages before each warp's stretch
  mine = warp_sum(mine);
  if (lane == 0) s_warp[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    const int w = s_warp[lane];
    const int wi = warp_scan_incl(w);
    s_warp[lane] = wi - w;
    if (lane == 31) s_total = wi;
  }
  __syncthreads();
  if (total > s_total) {
    if (threadIdx.x == 0) set_device_error(err, RPP_DERR_FULL);
    return;
  }
  // the k-th free page goes to the sequence whose scanned needs hold k
  int rank0 = s_warp[warp];
  for (int p0 = st.x; p0 < st.y && rank0 < total; p0 += 128) {
    const int p = p0 + 4 * lane;
    const int4 r = p < st.y ? load_refs4(refs, p, d.pages) : make_int4(-1, -1, -1, -1);
    const int have = (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    const int incl = warp_scan_incl(have);
    int rank = rank0 + incl - have;
    const int rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (rr[e] != 0) continue;
      if (rank < total) {
        int lo = 0, hi = n - 1;   // the last i with s_need[i] <= rank
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_need[mid] <= rank) lo = mid;
          else hi = mid - 1;
        }
        const int s = slots[lo];
        const int first = kFork ? lens[counts_or_from[lo]] / d.page_size : used_pages(lens[s], d.page_size);
        table[static_cast<long long>(s) * d.max_pages + first + (rank - s_need[lo])] = p + e;
        refs[p + e] = kFork ? 1 + shares * kForkShare : 1;
      }
      ++rank;
    }
    rank0 += __shfl_sync(0xffffffffu, incl, 31);
  }
  __syncthreads();   // every length is read before it is moved on
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int s = slots[i];
    if constexpr (kFork) {
      const int len = lens[counts_or_from[i]];
      lens[s] = len;
      if (len >= d.page_size) table[static_cast<long long>(s) * d.max_pages] = kForkMark;
    } else {
      lens[s] += counts_or_from[i];
    }
  }
}

// The scale bytes of a cache of 8-bit codes, [layers, pages, 2 * kv heads, page rows >> shift]; no array for one of 16-bit
// values.
struct PageScales {
  uint8_t* scales;
  int shift;
};

// The shared part of each fork (table entries, reference counts) and the rows of its own
// last page, in all layers.  blockIdx.x: pairs, grid-strided; blockIdx.y: shares of a pair's rows.  A pair's copy is
// r rows (those past the last whole page) of d * 2 bytes in each of layers * 2 * kv heads
// places; only those rows are moved.  What there is to do stands in the plan's marks, each taken away by
// who has done it, so a wrong page number in one source (recorded) leaves the other pairs alone,
// and a call that the plan refused finds no marks, whatever its lists and the state hold.
template <bool kScales>
__global__ void __launch_bounds__(kMoveThreads)
    kv_fork_copy_kernel(KvDims d, PageScales q, uint4* __restrict__ pool, int32_t* table,
                        const int32_t* lens, int32_t* refs, const int32_t* from,
                        const int32_t* to, int n, int32_t* err) {
  pdl_wait();
  pdl_trigger();
  const int vpr = d.head_dim / 8;                                   // 16-byte vectors of a row
  const long long page_vec = 2LL * d.kv_heads * d.page_size * vpr;  // of a page in one layer
  const long long layer_vec = page_vec * d.pages;
  const int head_vec = d.page_size * vpr;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int a = from[i], b = to[i];
    if (a < 0 || a >= d.slots || b < 0 || b >= d.slots) continue;   // (the same for all threads, as what follows)
    const int len = lens[b];
    if (!len_ok(len, d)) continue;
    const int full = len / d.page_size, rows = len % d.page_size;
    const int32_t* trow_from = table + static_cast<long long>(a) * d.max_pages;
    int32_t* trow_to = table + static_cast<long long>(b) * d.max_pages;
    const int pa = rows ? trow_from[full] : -1, pb = rows ? trow_to[full] : -1;
    const bool share = blockIdx.y == 0 && full > 0 && trow_to[0] == kForkMark;
    const bool copy = pb >= 0 && pb < d.pages && refs[pb] >= kForkShare;
    __syncthreads();   // the marks are read
    if (share) {
      for (int j = threadIdx.x; j < full; j += blockDim.x) {
        const int p = trow_from[j];
        trow_to[j] = p;
        if (p >= 0 && p < d.pages) atomicAdd(&refs[p], 1);
        else set_device_error(err, RPP_DERR_PAGE);
      }
    }
    if (!copy) continue;
    if (pa < 0 || pa >= d.pages) {
      if (threadIdx.x == 0) {
        set_device_error(err, RPP_DERR_PAGE);
        atomicSub(&refs[pb], kForkShare);
      }
      continue;
    }
    const uint4* src = pool + pa * page_vec;
    uint4* dst = pool + pb * page_vec;
    const int run = rows * vpr;                                     // contiguous vectors of one head
    const int groups = d.layers * 2 * d.kv_heads;
    const long long total = static_cast<long long>(groups) * run;
    const long long step = static_cast<long long>(gridDim.y) * kMoveThreads;
    constexpr int U = 4;
    for (long long v0 = static_cast<long long>(blockIdx.y) * kMoveThreads + threadIdx.x; v0 < total; v0 += U * step) {
      uint4 x[U];
      long long at[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long v = v0 + u * step;
        at[u] = -1;
        if (v < total) {
          const unsigned g = static_cast<unsigned long long>(v) <= 0xffffffffull
                                 ? static_cast<unsigned>(v) / static_cast<unsigned>(run)
                                 : static_cast<unsigned>(v / run);
          const unsigned layer = g / (2u * d.kv_heads), kh = g - layer * 2u * d.kv_heads;
          at[u] = layer * layer_vec + static_cast<long long>(kh) * head_vec + (v - static_cast<long long>(g) * run);
          x[u] = src[at[u]];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (at[u] >= 0) dst[at[u]] = x[u];
    }
    if constexpr (kScales) {   // of the blocks that these rows begin
      const int head = d.page_size >> q.shift, begun = ((rows - 1) >> q.shift) + 1;
      const long long page = 2LL * d.kv_heads * head, layer = page * d.pages;
      const long long bytes = static_cast<long long>(groups) * begun;
      for (long long v = static_cast<long long>(blockIdx.y) * kMoveThreads + threadIdx.x; v < bytes; v += step) {
        const long long g = v / begun, l = g / (2 * d.kv_heads);
        const long long at = l * layer + (g - l * 2 * d.kv_heads) * head + (v - g * begun);
        q.scales[pb * page + at] = q.scales[pa * page + at];
      }
    }
    if (threadIdx.x == 0) atomicSub(&refs[pb], kForkShare);
  }
}

// ---------------------------------------------------------------- free
// A CTA takes slots blockIdx.x, + gridDim.x, ...; each CTA checks the whole list first, so
// a slot out of range or given twice stops all of them before anything is changed.
__global__ void __launch_bounds__(kMoveThreads)
    kv_free_kernel(KvDims d, int32_t* table, int32_t* lens, int32_t* refs,
                   const int32_t* slots, int n, int32_t* err) {
  extern __shared__ uint32_t s_seen[];
  __shared__ Gate gate;
  pdl_wait();
  pdl_trigger();
  const int first = static_cast<int>(threadIdx.x) < n ? slots[threadIdx.x] : 0;
  if (!pass(slots, n, first, d, s_seen, &gate, err)) return;
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int s = slots[i];
    const int len = lens[s];
    if (!len_ok(len, d)) {
      if (threadIdx.x == 0) set_device_error(err, RPP_DERR_LENGTH);
      continue;
    }
    const int used = used_pages(len, d.page_size);
    int32_t* row = table + static_cast<long long>(s) * d.max_pages;
    for (int j = threadIdx.x; j < d.max_pages; j += blockDim.x) {
      if (j < used) {
        const int p = row[j];
        if (p < 0 || p >= d.pages) {
          set_device_error(err, RPP_DERR_PAGE);
        } else if (atomicSub(&refs[p], 1) <= 0) {   // was not in use: put back what was taken
          atomicAdd(&refs[p], 1);
          set_device_error(err, RPP_DERR_PAGE);
        }
      }
      row[j] = -1;
    }
    __syncthreads();   // every thread has read the length
    if (threadIdx.x == 0) lens[s] = 0;
  }
}

// ---------------------------------------------------------------- append
// Writes the K and V rows of the last tokens of each sequence (one layer): token t of
// sequence i, the j-th of its cnt, goes to position lens[slots[i]] - cnt + j.  A CTA takes
// tiles of kTok consecutive rows: their destinations first (one thread a row), then a flat
// 16-byte copy.
constexpr int kMaxTok = 32;
__global__ void __launch_bounds__(kMoveThreads)
    kv_append_kernel(KvDims d, uint4* __restrict__ pool_layer, const int32_t* table,
                     const int32_t* lens, const int32_t* refs, const uint4* k,
                     const uint4* v, int row_vec, const int32_t* slots,
                     const int32_t* cu, int n, int rows_max, int tok, int32_t* err) {
  extern __shared__ uint32_t s_seen[];
  __shared__ Gate gate;
  __shared__ long long s_at[kMaxTok];   // first vector of the row in the pool (head 0 of K), -1: none
  pdl_wait();
  pdl_trigger();
  const int first = static_cast<int>(threadIdx.x) < n ? slots[threadIdx.x] : 0;
  const int T = cu ? cu[n] : n, start = cu ? cu[0] : 0;
  const bool mine = cu && static_cast<int>(threadIdx.x) < n;
  const int c0 = mine ? cu[threadIdx.x] : 0, c1 = mine ? cu[threadIdx.x + 1] : 0;
  if (!pass(slots, n, first, d, s_seen, &gate, err, cu, c0, c1)) return;
  if (start < 0 || T > rows_max) {
    if (threadIdx.x == 0) set_device_error(err, RPP_DERR_ROWS);
    return;
  }
  const int vpr = d.head_dim / 8;
  const int head_vec = d.page_size * vpr;
  const long long page_vec = 2LL * d.kv_heads * head_vec;
  const int half = d.kv_heads * vpr;    // vectors of a K (or V) row
  const int tiles = (T + tok - 1) / tok;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int t0 = tile * tok;
    const int cnt_rows = min(tok, T - t0);
    if (static_cast<int>(threadIdx.x) < cnt_rows) {
      const int t = t0 + threadIdx.x;
      int i = t;
      long long back = 1;               // the row's sequence, and how far from its end (1: the last token)
      if (cu) {
        int lo = 0, hi = n - 1;         // the last i with cu[i] <= t (sequences without rows are passed over)
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (cu[mid] <= t) lo = mid;
          else hi = mid - 1;
        }
        i = lo;
        back = t < cu[i] ? 0 : static_cast<long long>(cu[i + 1]) - t;   // rows before cu[0] are nobody's
      }
      const int s = slots[i];
      const int len = lens[s];
      long long at = -1;
      if (!len_ok(len, d) || back < 1 || back > len) {
        set_device_error(err, RPP_DERR_LENGTH);
      } else {
        const int pos = static_cast<int>(len - back);
        const int p = table[static_cast<long long>(s) * d.max_pages + pos / d.page_size];
        if (p < 0 || p >= d.pages || refs[p] != 1) set_device_error(err, RPP_DERR_PAGE);   // not its own page
        else at = p * page_vec + static_cast<long long>(pos % d.page_size) * vpr;
      }
      s_at[threadIdx.x] = at;
    }
    __syncthreads();
    const int per = 2 * half;
    const int total = cnt_rows * per;
    constexpr int U = 4;
    for (int v0 = threadIdx.x; v0 < total; v0 += U * kMoveThreads) {
      uint4 x[U];
      long long to[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int w = v0 + u * kMoveThreads;
        to[u] = -1;
        if (w < total) {
          const int r = w / per;
          int c = w - r * per;
          const int isv = c >= half;
          c -= isv ? half : 0;
          const int h = c / vpr;
          if (s_at[r] >= 0) {
            to[u] = s_at[r] + static_cast<long long>(isv * d.kv_heads + h) * head_vec + (c - h * vpr);
            x[u] = (isv ? v : k)[static_cast<long long>(t0 + r) * row_vec + c];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (to[u] >= 0) pool_layer[to[u]] = x[u];
    }
    __syncthreads();   // s_at is rewritten for the next tile
  }
}

// ---------------------------------------------------------------- compact
// With `live` pages in use, the k-th page in use at or above `live` moves to the k-th free
// page below it.  moves[0] = their number (-1: the error word was set), moves[1] = live, then (to, from)
// pairs; remap[p] = the page's new number (-1: not in use).
__global__ void __launch_bounds__(kPlanThreads)
    kv_compact_plan_kernel(int pages, const int32_t* refs, int32_t* remap,
                           int32_t* live_out, int32_t* moves, const int32_t* err) {
  __shared__ int s_flag, s_live, s_low;
  __shared__ int s_warp[kPlanWarps];
  pdl_wait();
  pdl_trigger();
  if (quit(err, &s_flag)) {
    if (threadIdx.x == 0) moves[0] = -1;
    return;
  }
  const int warp = warp_id(), lane = lane_id();
  const int2 st = warp_stretch(pages);
  int mine = 0;
  for (int p = st.x + 4 * lane; p < st.y; p += 128) {
    const int4 r = load_refs4(refs, p, pages);
    mine += (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
  }
  mine = warp_sum(mine);
  if (lane == 0) s_warp[warp] = mine;
  __syncthreads();
  if (warp == 0) {
    const int w = s_warp[lane];
    const int wi = warp_scan_incl(w);
    s_warp[lane] = wi - w;
    if (lane == 31) s_live = wi;
  }
  if (threadIdx.x == 0) s_low = 0;
  __syncthreads();
  const int live = s_live;
  // pages in use below `live`: whole stretches before it, and the part of the one it lies in
  if (live > st.x) {
    int low = 0;
    const int end = min(st.y, live);
    for (int p = st.x + lane; p < end; p += 32) low += refs[p] > 0;
    low = warp_sum(low);
    if (lane == 0 && low) atomicAdd(&s_low, low);
  }
  __syncthreads();
  const int low = s_low;
  const int n_moves = live - low;
  if (threadIdx.x == 0) {
    moves[0] = n_moves;
    moves[1] = live;
    live_out[0] = live;
  }
  int2* pairs = reinterpret_cast<int2*>(moves + 2);
  int before = s_warp[warp];   // pages in use before the chunk
  for (int p0 = st.x; p0 < st.y; p0 += 128) {
    const int p = p0 + 4 * lane;
    const int4 r = p < st.y ? load_refs4(refs, p, pages) : make_int4(-1, -1, -1, -1);
    const int have = (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0);
    const int incl = warp_scan_incl(have);
    int k = before + incl - have;
    const int rr[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int q = p + e;
      if (q >= st.y) break;
      if (rr[e] > 0) {
        if (q >= live) pairs[k - low].y = q;
        else remap[q] = q;
        ++k;
      } else {
        if (q < live) pairs[q - k].x = q;   // the (q - k)-th page below `live` that is not in use
        remap[q] = -1;
      }
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  __syncthreads();
  for (int k = threadIdx.x; k < n_moves; k += kPlanThreads) remap[pairs[k].y] = pairs[k].x;
}

// Moves the pages, and writes the table and the reference counts by the new numbers
// (table_out and refs_out may be the arrays read).  A unit of the copy is 16 KB of a page
// in one layer (or what is left of it): four 16-byte vectors a thread in flight.
template <bool kScales>
__global__ void __launch_bounds__(kMoveThreads)
    kv_compact_move_kernel(KvDims d, PageScales q, uint4* __restrict__ pool, const int32_t* table,
                           const int32_t* lens, const int32_t* refs, int32_t* table_out,
                           int32_t* refs_out, const int32_t* remap, const int32_t* moves,
                           int32_t* err) {
  pdl_wait();
  pdl_trigger();
  // The plan's word, not the error word: this launch's own CTAs may set that, for a corrupt table, and
  // the pages of the other sequences have to move all the same, as the table says they did.
  const int n_moves = moves[0];
  if (n_moves < 0) return;
  const long long tid = static_cast<long long>(blockIdx.x) * kMoveThreads + threadIdx.x;
  const long long threads = static_cast<long long>(gridDim.x) * kMoveThreads;
  const int2* pairs = reinterpret_cast<const int2*>(moves + 2);
  const long long page_vec = 2LL * d.kv_heads * d.page_size * (d.head_dim / 8);
  const long long layer_vec = page_vec * d.pages;
  constexpr int U = 4;
  const int subs = static_cast<int>((page_vec + U * kMoveThreads - 1) / (U * kMoveThreads));
  const long long units = static_cast<long long>(n_moves) * d.layers * subs;
  for (long long w = blockIdx.x; w < units; w += gridDim.x) {
    const long long ml = w / subs;
    const int sub = static_cast<int>(w - ml * subs);
    const int k = static_cast<int>(ml / d.layers), layer = static_cast<int>(ml - static_cast<long long>(k) * d.layers);
    const int2 pr = pairs[k];
    const uint4* src = pool + layer * layer_vec + pr.y * page_vec;
    uint4* dst = pool + layer * layer_vec + pr.x * page_vec;
    const long long o = static_cast<long long>(sub) * U * kMoveThreads + threadIdx.x;
    uint4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (o + u * kMoveThreads < page_vec) x[u] = src[o + u * kMoveThreads];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (o + u * kMoveThreads < page_vec) dst[o + u * kMoveThreads] = x[u];
    if constexpr (kScales) {
      if (sub == 0) {
        const int bytes = 2 * d.kv_heads * (d.page_size >> q.shift);   // of a page in one layer
        const uint8_t* a = q.scales + (static_cast<long long>(layer) * d.pages + pr.y) * bytes;
        uint8_t* b = q.scales + (static_cast<long long>(layer) * d.pages + pr.x) * bytes;
        if (bytes % 4 == 0) {
          for (int e = threadIdx.x; e < bytes / 4; e += kMoveThreads)
            reinterpret_cast<uint32_t*>(b)[e] = reinterpret_cast<const uint32_t*>(a)[e];
        } else {
          for (int e = threadIdx.x; e < bytes; e += kMoveThreads) b[e] = a[e];
        }
      }
    }
  }
  const long long entries = static_cast<long long>(d.slots) * d.max_pages;
  for (long long e = tid; e < entries; e += threads) {
    const int s = static_cast<int>(e / d.max_pages), j = static_cast<int>(e - static_cast<long long>(s) * d.max_pages);
    const int len = lens[s];
    int to = -1;
    if (!len_ok(len, d)) {
      if (j == 0) set_device_error(err, RPP_DERR_LENGTH);
    } else if (j < used_pages(len, d.page_size)) {
      const int p = table[e];
      if (p >= 0 && p < d.pages) to = remap[p];
      if (to < 0) set_device_error(err, RPP_DERR_PAGE);
    }
    table_out[e] = to;
  }
  for (long long p = tid; p < d.pages; p += threads) {
    const int r = remap[p];
    if (r == p) {
      refs_out[p] = refs[p];
    } else if (r < 0 && p >= moves[1]) {   // free, and above the pages in use
      refs_out[p] = 0;
    }
  }
  for (long long k = tid; k < n_moves; k += threads) {
    const int2 pr = pairs[k];
    refs_out[pr.x] = refs[pr.y];
    refs_out[pr.y] = 0;
  }
}

}  // namespace

cudaError_t launch_kv_reserve(const KvDims& d, const KvState& c, const int32_t* slots, const int32_t* counts, int n,
                              int32_t* err, cudaStream_t stream) {
  const size_t smem = (static_cast<size_t>(n) + 1 + (d.slots + 31) / 32) * 4;
  return launch_pdl(kv_reserve_kernel<false>, dim3(1), dim3(kPlanThreads), smem, stream, d, c.table, c.lens, c.refs,
                    slots, counts, n, 0, err);
}

// the sizes that the copies of 16-bit rows see
inline KvDims as_16_bit(const KvDims& d, const Kv8Scales* q) {
  KvDims r = d;
  if (q) r.head_dim = d.head_dim / 2;
  return r;
}
inline PageScales page_scales(const Kv8Scales* q) { return q ? PageScales{q->scales, q->shift} : PageScales{nullptr, 0}; }

cudaError_t launch_kv_fork(const KvDims& dims, const KvState& c, const Kv8Scales* q, const int32_t* from,
                           const int32_t* to, int n, int32_t* err, cudaStream_t stream) {
  const KvDims d = as_16_bit(dims, q);
  // More CTAs than fit at once: the pairs' last pages are full to different degrees, and a share of
  // an empty one costs a CTA's start only.  16 prompts forked 8 times over 12 layers, with the free
  // before it: 73 us at 8 CTAs an SM, 66.6 at 16, 66.4 at 32, 75 at 64, 93 at 128; 4 forked twice 13.6 at each.
  const long long vec = static_cast<long long>(d.layers) * 2 * d.kv_heads * (d.page_size - 1) * (d.head_dim / 8);
  const int x = blocks_for(n, 32 * num_sms());
  const int most = (32 * num_sms() + x - 1) / x;
  const int y = blocks_for(vec / (4 * kMoveThreads) + 1, most < kMostShares ? most : kMostShares);
  const size_t smem = (static_cast<size_t>(n) + 1 + (d.slots + 31) / 32) * 4;
  const cudaError_t e = launch_pdl(kv_reserve_kernel<true>, dim3(1), dim3(kPlanThreads), smem, stream, d, c.table,
                                   c.lens, c.refs, to, from, n, y, err);
  if (e != cudaSuccess) return e;
  return launch_pdl(q ? kv_fork_copy_kernel<true> : kv_fork_copy_kernel<false>, dim3(x, y), dim3(kMoveThreads), 0, stream,
                    d, page_scales(q), static_cast<uint4*>(c.pool), c.table, static_cast<const int32_t*>(c.lens), c.refs, from, to, n, err);
}

cudaError_t launch_kv_free(const KvDims& d, const KvState& c, const int32_t* slots, int n, int32_t* err,
                           cudaStream_t stream) {
  const size_t smem = static_cast<size_t>((d.slots + 31) / 32) * 4;
  return launch_pdl(kv_free_kernel, dim3(blocks_for(n, 4 * num_sms())), dim3(kMoveThreads), smem, stream, d, c.table,
                    c.lens, c.refs, slots, n, err);
}

cudaError_t launch_kv_append(const KvDims& d, const KvState& c, int layer, const void* k, const void* v,
                             int row_stride, const int32_t* slots, const int32_t* cu, int n, int rows_max,
                             int32_t* err, cudaStream_t stream) {
  const size_t smem = static_cast<size_t>((d.slots + 31) / 32) * 4;
  const long long layer_vec = 2LL * d.kv_heads * d.page_size * (d.head_dim / 8) * d.pages;
  // rows a tile: enough CTAs for the grid first, then enough rows for the list check to pay
  int tok = (rows_max + 4 * num_sms() - 1) / (4 * num_sms());
  tok = tok < 1 ? 1 : tok > kMaxTok ? kMaxTok : tok;
  const int grid = blocks_for((static_cast<long long>(rows_max) + tok - 1) / tok, 8 * num_sms());
  return launch_pdl(kv_append_kernel, dim3(grid), dim3(kMoveThreads), smem, stream, d,
                    static_cast<uint4*>(c.pool) + layer * layer_vec, static_cast<const int32_t*>(c.table),
                    static_cast<const int32_t*>(c.lens), static_cast<const int32_t*>(c.refs),
                    static_cast<const uint4*>(k), static_cast<const uint4*>(v), row_stride / 8, slots, cu, n, rows_max,
                    tok, err);
}

cudaError_t launch_kv_compact(const KvDims& dims, const KvState& c, const Kv8Scales* q, int32_t* table_out,
                              int32_t* refs_out, int32_t* remap, int32_t* live, int32_t* moves, int32_t* err,
                              cudaStream_t stream) {
  const KvDims d = as_16_bit(dims, q);
  cudaError_t e = launch_pdl(kv_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, d.pages,
                             static_cast<const int32_t*>(c.refs), remap, live, moves, static_cast<const int32_t*>(err));
  if (e != cudaSuccess) return e;
  return launch_pdl(q ? kv_compact_move_kernel<true> : kv_compact_move_kernel<false>, dim3(8 * num_sms()),
                    dim3(kMoveThreads), 0, stream, d, page_scales(q), static_cast<uint4*>(c.pool), static_cast<const int32_t*>(c.table),
                    static_cast<const int32_t*>(c.lens), static_cast<const int32_t*>(c.refs), table_out, refs_out,
                    static_cast<const int32_t*>(remap), static_cast<const int32_t*>(moves), err);
}

}  // namespace rpp
