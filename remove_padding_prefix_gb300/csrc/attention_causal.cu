// Causal attention over packed prompts of different lengths, grouped heads, head size 64 or
// 128, fp16 or bf16, on the 5th-generation tensor cores:
//   o_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j    inside each sequence,
// query head h with the keys and values of kv head h / (nh / nkv).
//
// A work item is (sequence, query head, tile of 128 queries), run against 128-key tiles of K and
// V, the diagonal tile last.  A stream of items is 256 threads and half of tensor memory; an SM has two,
// so that while one's softmax runs the tensor cores have the other's products.  At d = 128, where a
// kv head has an even number of query heads, the two are one CTA's and take the two heads of a pair over
// one ring of K and V tiles: a tile then costs one write into shared memory for two products.
// Shared memory is the narrowest place at d = 128: S reads 64 KB a tile, PV 32 KB, and the
// tile itself is 64 KB, 1280 cycles of 128 bytes in all against 1024 of the tensor cores; 1024
// each where two share it.  Else the streams are CTAs of their own.
//
//   warp 0      TMA: the item's Q tile, then K_0 V_0 K_1 V_1 ... through a ring of tiles.
//   warp 1      issues S = Q K^T (M = 128, N = 128) into tensor memory and O += P V with P from tensor
//               memory, the first half of P's keys as soon as it is there.
//               d = 128: S and O fill the stream's 256 columns, so P takes the place of S and the
//               order is PV(j), S(j + 1).  d = 64: P has columns of its own and S(j + 1) is issued
//               once the scores of S(j) have been read.  S(0) of the next item follows the same way.
//   warps 2, 3  look over the V tiles that reach past the item's first query (below).
//   warps 4-7   softmax, one thread a query row, all 128 scores of a tile in registers (the
//               other warps give up registers for that): no exchange between threads.
//               Running maximum moved only when it grows by more than 8 (log2 units), so
//               P <= 2^8 (fp16: 2^15) and O is rarely rescaled; fp32 sum of the unrounded weights.  A diagonal
//               tile goes block by block, those of 32 keys that none of a warp's queries sees are
//               passed over.  At the end O / sum goes to the output row.
//
// Measured (bf16, one GB300): 8192 and 7 thousand tokens, 32 heads on 8 kv heads, d = 128: 720 us, 1480
// TFLOP/s, 0.79 of the measured cuBLAS burst.  64 prompts of 32 to 384, 16 heads, d = 64: 41.5 us against 16 us
// of reading and writing once: a softmax warp's item is some 1500 instructions that wait for one another, and
// tensor memory has room for two such chains an SM; four, with 64-key tiles, took as long.  8 prompts of
// 4096, 16 heads, d = 64: 351 us, 0.42 of the burst, by the same chain: a tile is half the products of d = 128
// for as many weights (tensor pipe 32%, exponentials 31%, issue slots 46% over one such prompt).
//
// P goes into its product in the type of the inputs, as the tensor cores take it: off by up to half a step of
// each weight (2^-8 of it in bf16, 2^-11 in fp16), as in the library's other attention.  A second product
// for what the rounding left, as in attention_decode.cu, would be half as many products again, and they
// bound long prompts.  The sum of the weights is of the unrounded ones.
//
// Items are taken longest first: with causal masking the cost of a query tile is its place
// in its sequence, so the list is by falling place, all sequences long enough and all
// heads at each (the heads of a kv head side by side: their K and V come from L2).
// One thread goes through the ceil(max_len / 128) places, so a max_len far above the lengths costs time: the
// 64 prompts above 86 us with 131072 and 140 with 262144, where the list is also too large for two single streams an SM.
// Every CTA builds the same list from cu_seqlens in its prologue and walks it there and back
// (item r CTAs + c in even rounds, r CTAs + CTAs - 1 - c in odd ones), which evens out the fall
// of the costs without a counter in memory.
//
// What a row must not see stays out of it: scores past the row become -inf before the
// maximum.  P is 0 there, but 0 * inf is not, so in the tiles on the diagonal V rows past
// the sequence are zeroed in shared memory, and elements of V that are not finite are
// taken out before the product; the outputs of the rows that see them are written from V once
// more (their sums with positive weights are the elements themselves), and so are outputs that a weight
// of 0 times an infinity in an earlier tile made NaN.  Two warps look over every V tile before the product may
// read it, so their wait on a ring slot is never a phase off.  Every mbarrier wait is bounded; a
// wait that gives up records RPP_DERR_TIMEOUT and the CTA drains, frees tensor memory
// and exits.
#include <algorithm>

#include "attention_common.cuh"
#include "nonfinite.cuh"

namespace rpp {

namespace {

using attn::neg_inf;
using attn::pack2;
using attn::tc_mma_f16_tmem_a;

constexpr int kT = 128;                  // queries of an item, keys of a tile
constexpr int kMaxPrompts = 4096;        // sequences of a call (their bounds are held in shared memory)
constexpr int kMaxCausalLen = 262144;    // tokens of a sequence (its tile counts are held there too)

// PAIR (d = 128 only): a CTA runs two streams of items side by side, the heads 2 i and 2 i + 1 of one kv head, over one ring
// of K and V tiles; else one stream, and two CTAs an SM.  A stream has 256 threads and 256 columns of
// tensor memory either way.
template <int D, bool PAIR>
struct Shape {
  static constexpr int kStreams = PAIR ? 2 : 1;
  static constexpr int kThreads = 256 * kStreams;          // a stream's warps 0-3: TMA, MMA, V's watch; 4-7: softmax
  static constexpr uint32_t kTmemCols = 256 * kStreams;
  static constexpr uint32_t kTileBytes = kT * D * 2;
  static constexpr bool kApart = D == 64;                  // P in columns of its own
  static constexpr int kQ = D == 64 ? 2 : 1;               // Q buffers of a stream
  // Ring of K / V tiles.  An even number, so that a slot is K's or V's for good: who waits for V tiles
  // only must not find a K tile's phase in between.
  static constexpr int kSlots = D == 64 || PAIR ? 4 : 2;
  static constexpr int kVSlots = kSlots / 2;               // V's, in turn
  static constexpr uint32_t kColP = kApart ? 192 : 0, kColO = 128;   // S at column 0 of the stream's
  static constexpr uint32_t kOffRing = kStreams * kQ * kTileBytes;
  static constexpr uint32_t kOffStage = kOffRing + kSlots * kTileBytes;   // 2 KB a softmax warp: rows on their way out
  static constexpr uint32_t kOffBar = kOffStage + kStreams * 4 * 2048;
  static constexpr uint32_t kOffMisc = kOffBar + kStreams * 32 * 8;
  static constexpr uint32_t kOffList = kOffMisc + 64;
};
// Registers: launched with 128 a thread, 32768 a stream (checked at the first launch: a split above
// what the launch has would wait for ever); 128 threads keep 80, the softmax's 128 take 176.  The compiler
// spills 20 to 48 bytes a thread in all.
constexpr int kLaunchRegs = 128, kLowRegs = 80, kHighRegs = 176;
static_assert(kLowRegs + kHighRegs == 2 * kLaunchRegs, "the split must be the launch's registers");

// The item list: in shared memory the sequences by falling number of items and, for each place i
// in a sequence, how many items lie at later places.
struct List {
  const int32_t* cu;      // [B + 1], in global memory
  const int16_t* perm;    // [sequences with an item]
  const int* first;       // [classes + 1]: first item at place i; [classes]: all items
  int classes, nh, total;
  float inv_nh;
};
__host__ __device__ constexpr uint32_t perm_bytes(int B) { return (static_cast<uint32_t>(B) * 2u + 15u) / 16u * 16u; }
__host__ __device__ constexpr uint32_t list_bytes(int B, int classes) {
  return perm_bytes(B) + static_cast<uint32_t>(classes + 1) * 4u;
}

struct CausalItem {
  int b, h, q0, c0, len;
  __device__ __forceinline__ int tiles() const { return q0 / kT + 1; }   // key tiles up to the diagonal
};

// A walk over the list by rising item number.  The place of an item in its sequence falls
// along the list, so after the first search it is a step or none.
struct Walk {
  const List& s;
  int place;
  __device__ __forceinline__ explicit Walk(const List& l) : s(l), place(-1) {}
  __device__ __forceinline__ void seek(int g) {
    if (place < 0) {                    // the smallest place with first[place] <= g
      int lo = 0, hi = s.classes - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s.first[mid] <= g) hi = mid;
        else lo = mid + 1;
      }
      place = lo;
    } else {
      while (place > 0 && s.first[place - 1] <= g) --place;
    }
  }
  __device__ __forceinline__ int tiles(int g) {   // of item g: nothing is divided
    seek(g);
    return place + 1;
  }
  __device__ __forceinline__ CausalItem at(int g) {
    CausalItem it;
    seek(g);
    it.q0 = place * kT;
    const int idx = g - s.first[place];
    int sq;
    if (idx < (1 << 23)) {              // exact in fp32, the quotient off by at most one
      sq = __float2int_rz(__int2float_rn(idx) * s.inv_nh);
      const int rest = idx - sq * s.nh;
      sq += rest >= s.nh ? 1 : rest < 0 ? -1 : 0;
    } else {
      sq = idx / s.nh;
    }
    it.b = s.perm[sq];
    it.h = idx - sq * s.nh;
    it.c0 = s.cu[it.b];
    it.len = s.cu[it.b + 1] - it.c0;
    return it;
  }
};

// Builds the list (all threads) at `base`, with classes + 1 words at `cursor` for the time of the call.
// False: the CTA must quit (error word set, or bad bounds, which are recorded).
__device__ __forceinline__ bool build_list(const int32_t* cu, int B, int T_max, int max_len, int nh,
                                           int classes, int32_t* err, int* s_status, uint8_t* base, int* cursor,
                                           List& out) {
  int16_t* perm = reinterpret_cast<int16_t*>(base);
  int* first = reinterpret_cast<int*>(base + perm_bytes(B));
  // cursor[c], c = 1 .. classes: sequences of c items, then the next position of one in perm
  if (threadIdx.x == 0) *s_status = device_error_set(err) ? -1 : 0;
  for (int c = threadIdx.x; c <= classes; c += blockDim.x) cursor[c] = 0;
  __syncthreads();
  if (*s_status) return false;
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    const int c0 = cu[b], c1 = cu[b + 1];
    const long long len = static_cast<long long>(c1) - c0;
    if (c0 < 0 || len < 0 || c1 > T_max || len > max_len) {
      atomicCAS(s_status, 0, len > max_len ? RPP_DERR_LENGTH : RPP_DERR_ROWS);
    } else if (len > 0) {
      atomicAdd(&cursor[(static_cast<int>(len) + kT - 1) / kT], 1);
    }
  }
  __syncthreads();
  if (*s_status) {
    if (threadIdx.x == 0 && *s_status > 0) set_device_error(err, *s_status);
    return false;
  }
  if (threadIdx.x == 0) {
    int longer = 0, items = 0;          // sequences with more items than the place, items at later places
    for (int i = classes - 1; i >= 0; --i) {
      const int n = cursor[i + 1];      // sequences with exactly i + 1 items
      cursor[i + 1] = longer;           // their first position in perm
      longer += n;
      first[i] = items;
      items += longer * nh;             // every sequence with more than i items has one at place i
    }
    first[classes] = items;
  }
  __syncthreads();
  if (threadIdx.x < 32) {               // a stable grouping by item count, the same in every CTA
    const int lane = threadIdx.x;
    for (int b0 = 0; b0 < B; b0 += 32) {
      const int b = b0 + lane;
      int c = 0;
      if (b < B) c = (cu[b + 1] - cu[b] + kT - 1) / kT;
      const unsigned peers = __match_any_sync(0xffffffffu, c);
      const int rank = __popc(peers & ((1u << lane) - 1u));
      if (c > 0) perm[cursor[c] + rank] = static_cast<int16_t>(b);
      __syncwarp();
      if (c > 0 && rank == 0) cursor[c] += __popc(peers);
      __syncwarp();
    }
  }
  __syncthreads();
  out = List{cu, perm, first, classes, nh, first[classes], __frcp_rn(static_cast<float>(nh))};
  return true;
}

// item number of round r for this CTA, -1 past the end: there and back over the list
__device__ __forceinline__ int item_of_round(int r, int total) {
  const int n = gridDim.x;
  const long long g = static_cast<long long>(r) * n + ((r & 1) ? n - 1 - static_cast<int>(blockIdx.x) : blockIdx.x);
  return g < total ? static_cast<int>(g) : -1;
}

// the word with the elements that are not finite set to zero
template <typename T>
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  const uint32_t f = nonfinite2<T>(w);
  return w & ~((f & 0x8000u ? 0xffffu : 0u) | (f & 0x80000000u ? 0xffff0000u : 0u));
}

__device__ __forceinline__ bool elect_one() {   // one lane of a converged warp
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Rewrites outputs from V's elements that are not finite, of the 32 rows from `own` on.  A whole warp, a lane with one
// of the rows (inv: one over its sum, nan: whether its output held NaN) and with D / 32 columns: it goes through V's
// rows in order, and a row's output in a column that has had such elements by then is their sum.  Where no
// sound row held NaN the tiles before the diagonal are in the outputs already, and the sum is of the diagonal tile's
// (noted: it has some) and added.  k, v, o: the first row of the sequence, len rows long, in the head's columns.
// A call, so that neither its code nor its registers are the kernel's (inlined: 512 prompts of 64 tokens, 32
// heads, d = 128, 7% more).
template <typename T, int D>
__device__ __noinline__ void sums_of_nonfinite(const T* k, const T* v, int kv_stride, T* o, long long pitch, int own,
                                               int len, float inv, bool nan, bool noted) {
  // rows whose sum is a number: all their scores are, or -inf (elsewhere the whole row is NaN)
  const bool number = inv > 0.f && inv < __int_as_float(0x7f800000) && own + static_cast<int>(lane_id()) < len;
  const uint32_t sound = __ballot_sync(0xffffffffu, number);
  const bool whole = __any_sync(0xffffffffu, nan && number);
  if (!whole && (!noted || !sound)) return;
  const int end = min(own + 32, len);
  constexpr int E = D / 32;                      // columns of a lane
  constexpr int U = 8;                           // rows at a time
  const int col = lane_id() * E;
  float sum[E] = {};
  uint32_t got = 0;                              // columns that have one
#pragma unroll 1
  for (int j0 = whole ? 0 : own / kT * kT; j0 < end; j0 += U) {   // own is a multiple of U
    uint32_t w[U][E / 2];
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int e = 0; e < E / 2; ++e)
        w[j][e] = j0 + j < end ? *reinterpret_cast<const uint32_t*>(v + static_cast<long long>(j0 + j) * kv_stride + col + 2 * e) : 0u;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      uint32_t bad = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) bad |= ((nonfinite2<T>(w[j][e / 2]) >> (16 * (e & 1) + 15)) & 1u) << e;
      if (__any_sync(0xffffffffu, bad != 0)) {
        // a K row that is not finite has the score -inf in a sound row: weight 0, and 0 * inf is NaN
        const bool none = __any_sync(0xffffffffu, part_nonfinite<T, D>(k + static_cast<long long>(j0 + j) * kv_stride + col));
#pragma unroll
        for (int e = 0; e < E; ++e)
          if ((bad >> e) & 1u) sum[e] += none ? __int_as_float(0x7fffffff) : half_of<T>(w[j][e / 2], e & 1);
        got |= bad;
      }
      if (j0 >= own && j0 + j < end && ((sound >> (j0 + j - own)) & 1u)) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if ((got >> e) & 1u) {
            T* at = o + (j0 + j) * pitch + col + e;
            *at = from_f32<T>(whole ? sum[e] : sum[e] + to_f32(*at));
          }
      }
    }
    // nothing changes a NaN any more: on to the warp's own rows (a sequence whose values are NaN all over)
    bool fixed = true;
#pragma unroll
    for (int e = 0; e < E; ++e) fixed = fixed && sum[e] != sum[e];
    if (j0 < own && __all_sync(0xffffffffu, fixed)) j0 = own - U;
  }
}

template <typename T, int D, bool PAIR>
__global__ void __launch_bounds__((Shape<D, PAIR>::kThreads), (PAIR ? 1 : 2))
    attention_causal_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                            const __grid_constant__ CUtensorMap tv, int q_x, int k_x, int v_x,
                            const T* k_rows, const T* v_rows, int kv_stride, const int32_t* cu, int B,
                            int T_max, int max_len, int nh, int group, int classes, T* __restrict__ out,
                            float scale_log2, int32_t* err) {
  using S = Shape<D, PAIR>;
  constexpr int HB = D / 64;                       // 64-column boxes of a row
  constexpr uint32_t kBox = kT * 128;              // bytes of one box: 128 rows of 128 bytes
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int xs = PAIR ? threadIdx.x >> 8 : 0;      // stream
  uint8_t* sQ = smem + xs * (S::kQ * S::kTileBytes);
  uint8_t* ring = smem + S::kOffRing;
  uint64_t* shared_bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t* bars = shared_bars + 32 * xs;
  uint64_t* full = shared_bars;                    // [kSlots] a ring tile has landed
  uint64_t* empty = shared_bars + 4;               // [kSlots] its last product (of each stream) is done
  uint64_t* q_full = bars + 8;                     // [kQ]
  uint64_t* q_empty = bars + 10;                   // [kQ] the item's last S is done
  uint64_t* s_full = bars + 12;                    // S computed (P over S: and every PV before it)
  uint64_t* s_free = bars + 13;                    // P apart: S read by the four warps
  uint64_t* p_half = bars + 14;                    // [2] half of P's keys written by the four warps
  uint64_t* pv_done = bars + 16;                   // P apart: O += P V done
  uint64_t* o_full = bars + 17;                    // the item's last PV is done
  uint64_t* o_free = bars + 18;                    // O read out by the four warps
  uint64_t* drain = bars + 19;
  uint64_t* v_ready = shared_bars + 20;            // [kSlots] a V tile has landed and been looked over
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 4);
  int* s_status = reinterpret_cast<int*>(smem + S::kOffMisc + 8);
  // [8] of the item of round r, in met[r % 8]: r + 1 where its diagonal V tile held an element that is not finite.
  // (The watch of V is at most three items ahead of the softmax, whose O has to be free for the next PV.)
  volatile int* met = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 32);
  const int warp = warp_id() & 7, lane = lane_id();   // warp of the stream

  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 8; ++i) met[i] = 0;
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], S::kStreams);
      mbar_init(&v_ready[i], 2);
    }
  }
  if ((threadIdx.x & 255) == 0) {
    for (int i = 0; i < S::kQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, 4);
    mbar_init(&p_half[0], 4);
    mbar_init(&p_half[1], 4);
    mbar_init(pv_done, 1);
    mbar_init(o_full, 1);
    mbar_init(o_free, 4);
    mbar_init(drain, 1);
    fence_mbarrier_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  List list;
  // (the list's scratch words lie where the tiles will be)
  if (!build_list(cu, B, T_max, max_len, nh / S::kStreams, classes, err, s_status, smem + S::kOffList, reinterpret_cast<int*>(smem),
                  list))
    return;
  if (item_of_round(0, list.total) < 0) return;    // the whole CTA; nothing allocated yet
  if (threadIdx.x < 32) {
    tmem_alloc(tmem_slot, S::kTmemCols);
    tmem_relinquish();
  }
  fence_proxy_async_smem();   // the list's scratch words come before the tiles that TMA writes there
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem0 = *tmem_slot, tmem = tmem0 + 256u * xs;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLowRegs));
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      if (lane == 0) {
        uint32_t idx = 0, nq = 0;                    // ring tiles and Q tiles issued
        bool ok = true;
        auto load = [&](const CUtensorMap* map, int col, int row) -> bool {
          const uint32_t s = idx % S::kSlots;
          if (!mbar_wait_bounded(&empty[s], ((idx / S::kSlots) & 1u) ^ 1u, abort_flag)) return false;
          mbar_arrive_expect_tx(&full[s], S::kTileBytes);
#pragma unroll
          for (int c = 0; c < HB; ++c)
            tma_load_2d(ring + s * S::kTileBytes + c * kBox, map, &full[s], col + 64 * c, row);
          ++idx;
          return true;
        };
        Walk walk(list);
        for (int r = 0; ok; ++r) {
          const int g = item_of_round(r, list.total);
          if (g < 0) break;
          CausalItem it = walk.at(g);
          it.h = it.h * S::kStreams + xs;
          const int kv_col = it.h / group * D;
          const int n = it.tiles();
          const uint32_t b = nq % S::kQ;
          if (!mbar_wait_bounded(&q_empty[b], ((nq / S::kQ) & 1u) ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&q_full[b], S::kTileBytes);
#pragma unroll
          for (int c = 0; c < HB; ++c)
            tma_load_2d(sQ + b * S::kTileBytes + c * kBox, &tq, &q_full[b], q_x + it.h * D + 64 * c, it.c0 + it.q0);
          ++nq;
          if (xs) continue;                            // the ring is stream 0's to fill
          for (int j = 0; j < n && ok; ++j)
            ok = load(&tk, k_x + kv_col, it.c0 + j * kT) && load(&tv, v_x + kv_col, it.c0 + j * kT);
        }
        if (!ok) {
          set_device_error(err, RPP_DERR_TIMEOUT);
          *abort_flag = 1;
        }
        // what is in flight lands before the CTA can exit: the last load of each buffer
        for (uint32_t i = idx > S::kSlots ? idx - S::kSlots : 0; i < idx; ++i)
          mbar_wait_bounded(&full[i % S::kSlots], (i / S::kSlots) & 1u, nullptr);
        for (uint32_t i = nq > S::kQ ? nq - S::kQ : 0; i < nq; ++i)
          mbar_wait_bounded(&q_full[i % S::kQ], (i / S::kQ) & 1u, nullptr);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp runs the loop and one elected lane issues, so that descriptors stay in uniform
      // registers: from a branch of one lane each product took 70 to 80 cycles to issue.
      {
        const bool leader = elect_one();
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
          const int w = mbar_wait_bounded(bar, parity, abort_flag) ? 1 : 0;
          return __all_sync(0xffffffffu, w) != 0;
        };
        constexpr int fmt = attn::Fmt<T>::v;
        constexpr uint32_t IDESC_S = idesc_f16(fmt, kT, kT);
        constexpr uint32_t IDESC_O = idesc_f16(fmt, kT, D) | (1u << 16);   // B (= V) N-major
        // V: N-major, 64 columns a box (the second box kBox further), 8 keys 1024 bytes apart
        constexpr uint64_t kVLead = D == 128 ? (static_cast<uint64_t>(kBox >> 4) << 16) - (1ull << 16) : 0ull;
        uint32_t ns = 0, np = 0, nq = 0, no = 0;     // S and PV issued, items whose S / PV are all issued
        bool ok = true;
        // A wait costs some 150 cycles even when there is nothing to wait for, so those for tiles that
        // came long ago are done while the softmax runs (the *_ready calls), and between its
        // signal and the products there is one wait.
        auto s_ready = [&](int j) -> bool {          // operands of the next S: tile j of its item
          const uint32_t i = 2u * ns, b = nq % S::kQ;
          return (j || wait(&q_full[b], (nq / S::kQ) & 1u)) && wait(&full[i % S::kSlots], (i / S::kSlots) & 1u);
        };
        auto do_s = [&](int j, int n) {
          const uint32_t s = 2u * ns % S::kSlots, b = nq % S::kQ;
          const uint32_t qa = smem_u32(sQ + b * S::kTileBytes), ka = smem_u32(ring + s * S::kTileBytes);
          if (leader) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              tc_mma_f16(tmem, sw128_kmajor_desc(qa + (k >> 2) * kBox) + 2u * (k & 3),
                         sw128_kmajor_desc(ka + (k >> 2) * kBox) + 2u * (k & 3), IDESC_S, k ? 1u : 0u);
            tc_commit(s_full);
            tc_commit(&empty[s]);
            if (j == n - 1) tc_commit(&q_empty[b]);
          }
          __syncwarp();
          ++ns;
          if (j == n - 1) ++nq;
        };
        auto pv_ready = [&](int j) -> bool {         // operands of the next PV but P, and its O
          return wait(&v_ready[(2u * np + 1u) % S::kSlots], (np / S::kVSlots) & 1u) &&
                 (j || !no || wait(o_free, (no - 1) & 1u));
        };
        auto do_pv = [&](int j, int n) -> bool {
          const uint32_t s = (2u * np + 1u) % S::kSlots;
          const uint64_t vd = sw128_kmajor_desc(smem_u32(ring + s * S::kTileBytes)) + kVLead;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!wait(&p_half[h], np & 1u)) return false;
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int k = 4 * h; k < 4 * h + 4; ++k)   // 16 keys: P columns +8, V +2048 bytes
                tc_mma_f16_tmem_a(tmem + S::kColO, tmem + S::kColP + 8u * k, vd + 128u * k, IDESC_O,
                                  (j | k) ? 1u : 0u);
              if (h) {
                tc_commit(&empty[s]);
                if (S::kApart) tc_commit(pv_done);
                if (j == n - 1) tc_commit(o_full);
              }
            }
            __syncwarp();
          }
          ++np;
          if (j == n - 1) ++no;
          return true;
        };
        // one line of tiles over this CTA's items; S runs one tile ahead of PV
        Walk walk(list);
        int rs = 0, js = 0, n_s = walk.tiles(item_of_round(0, list.total));
        int jp = 0, n_p = n_s;
        bool more = true;
        ok = s_ready(0);
        if (ok) {
          tc_fence_after();
          do_s(0, n_s);
        }
        while (ok) {
          // the tile after the one S was issued for last
          int j2 = js + 1, n2 = n_s;
          if (j2 == n_s) {
            const int g = item_of_round(++rs, list.total);
            more = g >= 0;
            j2 = 0;
            if (more) n2 = walk.tiles(g);
          }
          ok = (!more || s_ready(j2)) && pv_ready(jp);
          if (S::kApart && more) {
            ok = ok && wait(s_free, (ns - 1) & 1u);
            if (ok) {
              tc_fence_after();
              do_s(j2, n2);
            }
          }
          ok = ok && do_pv(jp, n_p);
          if (!S::kApart && more && ok) do_s(j2, n2);
          if (!more) break;
          jp = js = j2;
          n_p = n_s = n2;
        }
        if (!ok && leader) {
          set_device_error(err, RPP_DERR_TIMEOUT);
          *abort_flag = 1;
        }
        if (leader) tc_commit(drain);                // every MMA done before tensor memory is freed
        __syncwarp();
        mbar_wait_bounded(drain, 0, nullptr);
      }
    } else if (xs == 0) {
      // ------------------------------------------------------------ V: what some queries must not see
      // Every V tile passes here on its way to the product.  In a tile that reaches past the
      // item's first query, rows past the sequence become zero, and elements that are not finite
      // are taken out and the fact noted for the item.
      const int t = (warp - 2) * 32 + lane;
      uint32_t nv = 0;                               // V tiles passed
      bool ok = true;
      Walk walk(list);
      for (int r = 0; ok; ++r) {
        const int g = item_of_round(r, list.total);
        if (g < 0) break;
        const CausalItem it = walk.at(g);
        const int n = it.tiles();
        for (int j = 0; j < n; ++j, ++nv) {
          const uint32_t i = 2u * nv + 1u, s = i % S::kSlots;
          const int w = mbar_wait_bounded(&full[s], (i / S::kSlots) & 1u, abort_flag) ? 1 : 0;
          if (!__all_sync(0xffffffffu, w)) {
            ok = false;
            break;
          }
          if (j == n - 1) {
#pragma unroll 1
            for (int row = t; row < kT; row += 64) {
              uint8_t* vrow = ring + s * S::kTileBytes + row * 128;
              auto chunk = [&](int c) {
                return reinterpret_cast<uint4*>(vrow + (c >> 3) * kBox + ((c & 7) ^ (row & 7)) * 16);
              };
              if (j * kT + row >= it.len) {
#pragma unroll
                for (int c = 0; c < HB * 8; ++c) *chunk(c) = make_uint4(0u, 0u, 0u, 0u);
              } else {
                uint32_t f = 0;
#pragma unroll 4
                for (int c = 0; c < HB * 8; ++c) {
                  const uint4 x = *chunk(c);
                  f |= nonfinite2<T>(x.x) | nonfinite2<T>(x.y) | nonfinite2<T>(x.z) | nonfinite2<T>(x.w);
                }
                if (f & 0x80008000u) {
                  met[r & 7] = r + 1;
#pragma unroll 1
                  for (int c = 0; c < HB * 8; ++c) {
                    const uint4 x = *chunk(c);
                    *chunk(c) = make_uint4(finite2<T>(x.x), finite2<T>(x.y), finite2<T>(x.z), finite2<T>(x.w));
                  }
                }
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&v_ready[s]);
        }
      }
      if (!ok && lane == 0) {
        set_device_error(err, RPP_DERR_TIMEOUT);
        *abort_flag = 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kHighRegs));
    // ------------------------------------------------------------ softmax: one thread a query row
    const int quad = warp & 3;                     // tensor-memory lanes of this warp
    const uint32_t t_s = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t t_p = t_s + S::kColP, t_o = t_s + S::kColO;
    // a power of two from it on (2^127 at most)
    const float scale_up = __int_as_float(min((__float_as_int(scale_log2) + 0x7fffff) & 0x7f800000, 254 << 23));
    // fp16 weights (and so their sum and O) are kept 2^7 times as large, up to 2^15: below the smallest
    // step of fp16, 2^-24, a weight is lost, and a long sequence has many small ones.
    constexpr float kUp = std::is_same<T, __half>::value ? 7.f : 0.f;
    // A maximum is a rounded product, the weights' exponents come from an fma, whose product is not: they differ by up to
    // half a last place of the maximum, and that has to stay inside the weights' range.  From kFar on weights begin
    // lower and the maximum moves with every larger score; from kOne on two scores that differ are 16 or more apart, so
    // beside the largest one weights are below 2^-16 whatever the scale, and a scale that is a power of two (the
    // next one) makes the products exact.  Tests of scores of any size; 1.2% of the time of long prompts.
    constexpr float kFar = 0x1p22f, kOne = 0x1p28f;
    uint8_t* stage = smem + S::kOffStage + (4 * xs + quad) * 2048;
    uint32_t ns = 0, no = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      const int w = mbar_wait_bounded(bar, parity, abort_flag) ? 1 : 0;
      return __all_sync(0xffffffffu, w) != 0;
    };
    Walk walk(list);
    int g = item_of_round(0, list.total);            // >= 0 here
    auto item = [&](int i) {
      CausalItem t = walk.at(i);
      t.h = t.h * S::kStreams + xs;
      return t;
    };
    CausalItem it = item(g), nx = it;
    for (int r = 1; g >= 0; ++r, it = nx) {
      const int nt = it.tiles();
      const bool live = it.q0 + quad * 32 < it.len;   // some of this warp's queries exist
      float m = neg_inf(), l = 0.f;
      for (int j = 0; j < nt; ++j) {
        // 32-key blocks of the tile that this warp's queries see, in the diagonal tile the last in part
        const bool tri = j == nt - 1;
        const int seen = !live ? 0 : tri ? quad + 1 : kT / 32;
        if (!wait(s_full, ns & 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint64_t sum2[2] = {0ull, 0ull}, nm2 = 0ull, by2 = 0ull;
        // the last PV has read P and left O (P over S: s_full says so)
        auto last_pv = [&]() -> bool {
          if (!S::kApart || j == 0) return true;
          if (!wait(pv_done, (ns - 1) & 1u)) return false;
          tc_fence_after();
          return true;
        };
        // Takes the tile's maximum into the row's: it moves lazily, and then O and the sum with it.
        // The accesses to tensor memory are the whole warp's (factor 1 for the rows that stay).
        auto take_max = [&](float top) {
          const float mx = __fmul_rn(top, scale_log2);
          const bool move = mx > (fabsf(m) < kFar ? m + 8.0f : m);
          if (j == 0) {
            m = mx;
          } else if (__any_sync(0xffffffffu, move)) {
            const float alpha = move ? ex2_approx(m - mx) : 1.0f;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t ov[16];
              tmem_ld_32x32b_x16(t_o + 16 * c, ov);
              tmem_ld_wait_tied16(ov);
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              tmem_st_32x32b_x16(t_o + 16 * c, ov);
              tmem_st_wait_tied16(ov);
            }
            if (move) {
              l *= alpha;
              m = mx;
            }
          }
          // scores all -inf so far: weights 0, not 2^(-inf + inf)
          float nm = m == neg_inf() ? 0.f : kUp - m, by = scale_log2;
          if (fabsf(m) >= kFar && m != neg_inf()) {
            nm = (kUp > 0.f ? 4.f : 0.f) - m;
            if (fabsf(m) >= kOne) {
              by = scale_up;
              nm = mx < m ? neg_inf() : -top * by;
            }
          }
          nm2 = f2_pack(nm, nm);
          by2 = f2_pack(by, by);
        };
        auto weights = [&](const uint32_t* sc, uint32_t* p, int n2) {   // 2 n2 scores -> n2 pairs of weights
#pragma unroll
          for (int e = 0; e < n2; ++e) {
            const uint64_t x2 = f2_fma(f2_pack(__uint_as_float(sc[2 * e]), __uint_as_float(sc[2 * e + 1])), by2, nm2);
            const float p0 = ex2_approx(f2_lo(x2)), p1 = ex2_approx(f2_hi(x2));
            sum2[e & 1] = f2_add(sum2[e & 1], f2_pack(p0, p1));
            p[e] = pack2<T>(p0, p1);
          }
        };
        auto part_out = [&](int c) {                  // 64 keys of P are in tensor memory
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_half[c]);
        };
        auto s_read = [&]() {                         // S may be overwritten
          if (!S::kApart) return;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free);
        };
        if (seen == kT / 32 && !tri) {
          // ---- a whole tile: scores in registers, the second part on its way while the first
          // part's maximum is taken
          uint32_t v[kT];
          float pm[4];
          auto load = [&](int c) {
            tmem_ld_32x32b_x32(t_s + 64 * c, v + 64 * c);
            tmem_ld_32x32b_x32(t_s + 64 * c + 32, v + 64 * c + 32);
          };
          load(0);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tmem_ld_wait_tied32(v + 64 * c);
            tmem_ld_wait_tied32(v + 64 * c + 32);
            if (c + 1 < 2) load(c + 1);
            else s_read();
            if (c == 0) {
#pragma unroll
              for (int t = 0; t < 4; ++t) pm[t] = fmaxf(__uint_as_float(v[t]), __uint_as_float(v[t + 4]));
            }
#pragma unroll
            for (int e = c ? 64 * c : 8; e < 64 * c + 64; e += 8)
#pragma unroll
              for (int t = 0; t < 4; ++t)
                pm[t] = max3(pm[t], __uint_as_float(v[e + t]), __uint_as_float(v[e + t + 4]));
          }
          if (!last_pv()) {
            ok = false;
            break;
          }
          take_max(fmaxf(max3(pm[0], pm[1], pm[2]), pm[3]));
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            weights(v + 64 * c, v + 32 * c, 32);
            tmem_st_32x32b_x32(t_p + 32 * c, v + 32 * c);
            tmem_st_wait_tied32(v + 32 * c);
            part_out(c);
          }
        } else {
          // ---- a tile that these queries see in part: block by block, twice (maximum, weights);
          // blocks that none of them sees have weight 0
          uint32_t v[32];
          auto block = [&](int c) {
            tmem_ld_32x32b_x32(t_s + 32 * c, v);
            tmem_ld_wait_tied32(v);
            if (tri && c == seen - 1) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e > lane) v[e] = 0xff800000u;
            }
          };
          float mx = neg_inf();
#pragma unroll 1
          for (int c = 0; c < seen; ++c) {
            block(c);
            float pm[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) pm[t] = fmaxf(__uint_as_float(v[t]), __uint_as_float(v[t + 4]));
#pragma unroll
            for (int e = 8; e < 32; e += 8)
#pragma unroll
              for (int t = 0; t < 4; ++t)
                pm[t] = max3(pm[t], __uint_as_float(v[e + t]), __uint_as_float(v[e + t + 4]));
            mx = fmaxf(mx, fmaxf(max3(pm[0], pm[1], pm[2]), pm[3]));
          }
          if (!last_pv()) {
            ok = false;
            break;
          }
          if (seen > 0) take_max(mx);
#pragma unroll 1
          for (int c = 0; c < kT / 32; ++c) {
            if (c < seen) {
              block(c);
              weights(v, v, 16);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) v[e] = 0u;
            }
            if (live) {
              tmem_st_32x32b_x16(t_p + 16 * c, v);
              tmem_st_wait_tied16(v);
            }
            if (c == kT / 32 - 1) s_read();
            if (c & 1) part_out(c >> 1);
          }
        }
        l += (f2_lo(sum2[0]) + f2_hi(sum2[0])) + (f2_lo(sum2[1]) + f2_hi(sum2[1]));
        ++ns;
      }
      g = item_of_round(r, list.total);
      if (g >= 0) nx = item(g);                      // while the last PV runs
      if (!ok || !wait(o_full, no & 1u)) {
        ok = false;
        break;
      }
      ++no;
      tc_fence_after();
      const float inv = __fdividef(1.0f, l);
      const uint64_t inv2 = f2_pack(inv, inv);
      // A thread has a row, a store wants whole lines: 32 columns at a time through 2 KB of shared
      // memory of the warp's own (16-byte chunk u of row r at u ^ (r / 2 & 3): no bank conflict
      // either way), then four lanes a row.  Rolled: every instruction here runs once or twice an item, and
      // fetching it is what that costs.
      const long long pitch = static_cast<long long>(nh) * D;
      const int rr = lane >> 2, ch = lane & 3;         // row of an 8-row group and chunk that this lane stores
      T* obase = out + (it.c0 + it.q0 + quad * 32 + rr) * pitch + it.h * D + 8 * ch;
      const int rows_left = it.len - it.q0 - quad * 32 - rr;
      uint64_t all2[2] = {0ull, 0ull};                 // sum of the row's outputs
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        tmem_ld_32x32b_x32(t_o + 32 * c, x);
        tmem_ld_wait_tied32(x);
        uint8_t* mine = stage + lane * 64;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t x2 = f2_mul(f2_pack(__uint_as_float(x[8 * u + 2 * e]), __uint_as_float(x[8 * u + 2 * e + 1])), inv2);
            w[e] = pack2<T>(f2_lo(x2), f2_hi(x2));
            all2[e & 1] = f2_add(all2[e & 1], x2);
          }
          *reinterpret_cast<uint4*>(mine + ((u ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          // (row 8 u + rr: its swizzle is that of rr, 8 u / 2 being a multiple of 4)
          const uint4 w = *reinterpret_cast<const uint4*>(stage + (8 * u + rr) * 64 + ((ch ^ ((rr >> 1) & 3)) << 4));
          if (8 * u < rows_left) *reinterpret_cast<uint4*>(obase + 8 * u * pitch + 32 * c) = w;
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
      // V elements that are not finite: a column that has one up to a row's own key is there the sum of such
      // elements, which needs neither weights nor the finite rest.  They were taken out of the diagonal tile (the
      // note is visible here: o_full came after the v_ready of that tile), and before it a weight that underflowed
      // to 0 made NaN of one (nonfinite.cuh), which the sum of the row's outputs shows.
      const float all = (f2_lo(all2[0]) + f2_hi(all2[0])) + (f2_lo(all2[1]) + f2_hi(all2[1]));
      const bool noted = met[(r - 1) & 7] == r, nan = all != all;
      if (live && (noted || (nt > 1 && __any_sync(0xffffffffu, nan)))) {
        const long long first = static_cast<long long>(it.c0) * kv_stride + it.h / group * D;
        sums_of_nonfinite<T, D>(k_rows + first, v_rows + first, kv_stride, out + static_cast<long long>(it.c0) * pitch + it.h * D,
                                pitch, it.q0 + quad * 32, it.len, inv, nan, noted);
      }
    }
    if (!ok && lane == 0) {
      set_device_error(err, RPP_DERR_TIMEOUT);
      *abort_flag = 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x < 32) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem0, S::kTmemCols);
  }
}

// The tensor maps of a call, and where the columns of q, k and v start in them.
struct Maps {
  CUtensorMap q, k, v;
  int q_x = 0, k_x = 0, v_x = 0;
};

template <typename T, int D, bool PAIR>
cudaError_t launch(const Maps& t, const CausalArgs& a, cudaStream_t stream) {
  using S = Shape<D, PAIR>;
  const int classes = (a.max_len + kT - 1) / kT;
  const size_t smem = 1024 + S::kOffList + list_bytes(a.B, classes);
  static SmemLimit limit;
  const cudaError_t e =
      limit.raise(attention_causal_kernel<T, D, PAIR>,
                  1024 + S::kOffList + list_bytes(kMaxPrompts, kMaxCausalLen / kT), kLaunchRegs);
  if (e != cudaSuccess) return e;
  // never more CTAs than items: ceil(len / 128) <= len / 128 + 1 for each sequence
  const long long most = (static_cast<long long>(a.T_max) / kT + a.B) * (a.nh / S::kStreams);
  const long long room = (PAIR ? 1LL : 2LL) * num_sms();
  const int grid = static_cast<int>(most < room ? most : room);
  return launch_pdl(attention_causal_kernel<T, D, PAIR>, dim3(grid), dim3(S::kThreads), smem, stream, t.q, t.k, t.v,
                    t.q_x, t.k_x, t.v_x, static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.kv_stride, a.cu, a.B, a.T_max, a.max_len, a.nh,
                    a.nh / a.nkv, classes, static_cast<T*>(a.out), a.scale * 1.4426950408889634f, a.err);
}

template <typename T>
cudaError_t dispatch(const Maps& t, const CausalArgs& a, cudaStream_t stream) {
  // Pairs of heads at d = 128, where a kv head has an even number of them.  Pairs against single streams, 32 heads
  // on 8 kv heads, d = 128: 621 / 740 us for two prompts of 8192 and 7500, 292 / 314 us for 32 of 1024, 142 / 129
  // us for 256 of 128, 210 / 217 us for 512 of 64.  At d = 64 shared memory is not the narrowest place: 16
  // heads on 4, 350 / 341 us for 8 of 4096, 61 / 60 us for 256 of 128.
  if (a.d == 64) return launch<T, 64, false>(t, a, stream);
  return (a.nh / a.nkv) % 2 == 0 ? launch<T, 128, true>(t, a, stream) : launch<T, 128, false>(t, a, stream);
}

}  // namespace

bool attention_causal_supported(int B, int max_len, int d) {
  return B <= kMaxPrompts && max_len <= kMaxCausalLen && (d == 64 || d == 128);
}

cudaError_t launch_attention_causal(const CausalArgs& a, cudaStream_t stream) {
  const CUtensorMapDataType dt =
      a.dtype == RPP_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  Maps t;
  // Columns of one projection's output: one map over all of them (encoding one takes about as
  // long on the host as the rest of the call before the launch).
  const uintptr_t q = reinterpret_cast<uintptr_t>(a.q), k = reinterpret_cast<uintptr_t>(a.k),
                  v = reinterpret_cast<uintptr_t>(a.v);
  const uintptr_t first = std::min(q, std::min(k, v));
  const uintptr_t end = std::max(q + 2u * static_cast<uintptr_t>(a.nh) * a.d,
                                 std::max(k, v) + 2u * static_cast<uintptr_t>(a.nkv) * a.d);
  // A map's row is a whole stride, whatever part of it is this tensor's: the boxes that are loaded
  // lie inside the heads' columns.
  auto map = [&](CUtensorMap* m, const void* base, int stride) {
    return make_tmap_2d(m, base, dt, 2, a.T_max, stride, kT, 64, CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (a.q_stride == a.kv_stride && end - first <= 2u * static_cast<uintptr_t>(a.q_stride)) {
    if (!map(&t.q, reinterpret_cast<const void*>(first), a.q_stride)) return cudaErrorInvalidValue;
    t.k = t.v = t.q;
    t.q_x = static_cast<int>((q - first) / 2);
    t.k_x = static_cast<int>((k - first) / 2);
    t.v_x = static_cast<int>((v - first) / 2);
  } else if (!map(&t.q, a.q, a.q_stride) || !map(&t.k, a.k, a.kv_stride) || !map(&t.v, a.v, a.kv_stride)) {
    return cudaErrorInvalidValue;
  }
  return a.dtype == RPP_F16 ? dispatch<__half>(t, a, stream) : dispatch<__nv_bfloat16>(t, a, stream);
}

}  // namespace rpp
