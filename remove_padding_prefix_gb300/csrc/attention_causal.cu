// Causal attention over packed prompts of different lengths, grouped heads, head size 64 or
// 128, fp16 or bf16, on the 5th-generation tensor cores:
//   o_i = sum_{j <= i} softmax_j(scale q_i . k_j) v_j    inside each sequence,
// query head h with the keys and values of kv head h / (nh / nkv).
//
// A work item is (sequence, query head, NQ tiles of 128 queries); one CTA at a time runs
// it against 128-key tiles of K and V, the diagonal tile of each query tile last.
//
//   warp 0       TMA: the item's Q tiles, then K_0 V_0 K_1 V_1 ... through a ring of tiles that
//                both query tiles read (NQ = 2: each K and V tile serves 256 queries, which
//                halves the shared-memory fill a product needs).
//   warp 1       one thread issues S = Q K^T (M = 128, N = 128) into tensor memory and O += P V
//                with P from tensor memory.  Per query tile the order is PV(j), S(j + 1): P
//                takes the place of S, tensor memory being full (NQ = 2: two S and two O tiles
//                are its 512 columns at d = 128).  With two query tiles one's products run
//                while the other's softmax does.  S(0) of the next item follows the last PV.
//   4 NQ warps   softmax, one thread a query row, all 128 scores of a tile in registers: no
//                exchange between threads.  Running maximum moved only when it grows by more
//                than 8 (log2 units), so P <= 2^8 and O is rarely rescaled; fp32 sum of the
//                unrounded weights.  Only the diagonal tile is masked.  At the end O / sum goes
//                to the output row.
//
// Items are taken longest first: with causal masking the cost of a query tile is its place
// in its sequence, so the list is by falling place, all sequences long enough and all
// heads at each (the heads of a kv head side by side: their K and V come from L2).
// Every CTA builds the same list from cu_seqlens in its prologue and walks it there and back
// (item r CTAs + c in even rounds, r CTAs + CTAs - 1 - c in odd ones), which evens out the fall
// of the costs without a counter in memory.
//
// What a row must not see stays out of it: scores past the row become -inf before the
// maximum.  P is 0 there, but 0 * inf is not, so in the diagonal tile V rows past the
// sequence are zeroed in shared memory, and elements of V that are not finite are
// taken out before the product and added back to the rows that may see them (their sums
// with positive weights are the elements themselves).  Every mbarrier wait is bounded; a
// wait that gives up records RPP_DERR_TIMEOUT and the CTA drains, frees tensor memory
// and exits.
#include <algorithm>

#include "attention_common.cuh"

namespace rpp {

namespace {

using attn::neg_inf;
using attn::pack2;
using attn::tc_mma_f16_tmem_a;

constexpr int kT = 128;                  // queries and keys of a tile
constexpr int kMaxPrompts = 4096;        // sequences of a call (their bounds are held in shared memory)
constexpr int kMaxCausalLen = 262144;    // tokens of a sequence (its tile counts are held there too)

template <int D, int NQ>
struct Shape {
  static constexpr uint32_t kTileBytes = kT * D * 2;
  static constexpr int kSlots = NQ == 2 ? (D == 128 ? 4 : 8) : (D == 128 ? 2 : 4);   // ring of K / V tiles
  static constexpr int kThreads = 64 + NQ * 128;
  static constexpr uint32_t kTmemCols = 256 * NQ;
  static constexpr uint32_t kColO = 128 * NQ;      // S of tile x at 128 x, O at kColO + 128 x (P over S)
  static constexpr uint32_t kOffRing = NQ * kTileBytes;
  static constexpr uint32_t kOffBar = kOffRing + kSlots * kTileBytes;
  static constexpr uint32_t kOffMisc = kOffBar + 32 * 8;
  static constexpr uint32_t kOffList = kOffMisc + 32;
};

// the item list in shared memory: cu_seqlens, sequences by falling number of items, and
// for each place i in a sequence how many items lie at later places
struct List {
  const int* cu;          // [B + 1]
  const int16_t* perm;    // [sequences with an item]
  const int* first;       // [classes + 1]: first item at place i; first[0] + its own = all
  int classes, nh, total;
};
__host__ __device__ constexpr uint32_t list_bytes(int B, int classes) {
  return (static_cast<uint32_t>(B + 1) * 4u + 15u) / 16u * 16u + (static_cast<uint32_t>(B) * 2u + 15u) / 16u * 16u +
         static_cast<uint32_t>(2 * classes + 3) * 4u;
}

struct CausalItem {
  int b, h, q0, c0, len;
};

template <int ROWS>
__device__ __forceinline__ CausalItem item_at(const List& s, int g) {
  int lo = 0, hi = s.classes - 1;       // the smallest place i with first[i] <= g
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (s.first[mid] <= g) hi = mid;
    else lo = mid + 1;
  }
  const int idx = g - s.first[lo];
  CausalItem it;
  const int sq = idx / s.nh;
  it.b = s.perm[sq];
  it.h = idx - sq * s.nh;
  it.q0 = lo * ROWS;
  it.c0 = s.cu[it.b];
  it.len = s.cu[it.b + 1] - it.c0;
  return it;
}

// Builds the list (all threads).  False: the CTA must quit (error word set, or bad bounds, which are recorded).
template <int ROWS>
__device__ __forceinline__ bool build_list(const int32_t* __restrict__ cu, int B, int T_max, int max_len, int nh,
                                           int classes, int32_t* err, int* s_status, uint8_t* base, List& out) {
  int* s_cu = reinterpret_cast<int*>(base);
  int16_t* perm = reinterpret_cast<int16_t*>(base + (static_cast<uint32_t>(B + 1) * 4u + 15u) / 16u * 16u);
  int* first = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(perm) +
                                      (static_cast<uint32_t>(B) * 2u + 15u) / 16u * 16u);
  int* cursor = first + classes + 2;    // [classes + 1]: by number of items: count, then next position in perm
  if (threadIdx.x == 0) *s_status = device_error_set(err) ? -1 : 0;
  for (int c = threadIdx.x; c <= classes; c += blockDim.x) cursor[c] = 0;
  for (int b = threadIdx.x; b <= B; b += blockDim.x) s_cu[b] = __ldg(cu + b);
  __syncthreads();
  if (*s_status) return false;
  __syncthreads();
  for (int b = threadIdx.x; b < B; b += blockDim.x) {
    const int c0 = s_cu[b], c1 = s_cu[b + 1];
    const long long len = static_cast<long long>(c1) - c0;
    if (c0 < 0 || len < 0 || c1 > T_max || len > max_len) {
      atomicCAS(s_status, 0, len > max_len ? RPP_DERR_LENGTH : RPP_DERR_ROWS);
    } else if (len > 0) {
      atomicAdd(&cursor[(static_cast<int>(len) + ROWS - 1) / ROWS], 1);
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
      if (b < B) c = (s_cu[b + 1] - s_cu[b] + ROWS - 1) / ROWS;
      const unsigned peers = __match_any_sync(0xffffffffu, c);
      const int rank = __popc(peers & ((1u << lane) - 1u));
      if (c > 0) perm[cursor[c] + rank] = static_cast<int16_t>(b);
      __syncwarp();
      if (c > 0 && rank == 0) cursor[c] += __popc(peers);
      __syncwarp();
    }
  }
  __syncthreads();
  out = List{s_cu, perm, first, classes, nh, first[classes]};
  return true;
}

// item number of round r for this CTA, -1 past the end: there and back over the list
__device__ __forceinline__ int item_of_round(int r, int total) {
  const int n = gridDim.x;
  const long long g = static_cast<long long>(r) * n + ((r & 1) ? n - 1 - static_cast<int>(blockIdx.x) : blockIdx.x);
  return g < total ? static_cast<int>(g) : -1;
}

// true where a 16-bit float of the word is not finite: bits of the low / high element
template <typename T>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
  constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
  return ((w & e) == e ? 0xffffu : 0u) | ((w & (e << 16)) == (e << 16) ? 0xffff0000u : 0u);
}

template <typename T, int D, int NQ>
__global__ void __launch_bounds__(Shape<D, NQ>::kThreads, NQ == 2 ? 1 : 2)
    attention_causal_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                            const __grid_constant__ CUtensorMap tv, int q_x, int k_x, int v_x,
                            const T* __restrict__ v_rows, int kv_stride,
                            const int32_t* __restrict__ cu, int B, int T_max, int max_len, int nh, int group,
                            int classes, T* __restrict__ out, float scale_log2, int32_t* err) {
  using S = Shape<D, NQ>;
  constexpr int ROWS = NQ * kT;
  constexpr int HB = D / 64;                       // 64-column boxes of a row
  constexpr uint32_t kBox = kT * 128;              // bytes of one box: 128 rows of 128 bytes
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* ring = smem + S::kOffRing;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t* full = bars;                           // [kSlots] a ring tile has landed
  uint64_t* empty = bars + 8;                      // [kSlots] its last product is done
  uint64_t* q_full = bars + 16;                    // [NQ]
  uint64_t* q_empty = bars + 18;                   // [NQ] the item's last S is done
  uint64_t* s_full = bars + 20;                    // [NQ] S computed (and every PV before it)
  uint64_t* p_full = bars + 22;                    // [NQ] P written by the tile's four warps
  uint64_t* o_full = bars + 24;                    // [NQ] the item's last PV is done
  uint64_t* o_free = bars + 26;                    // [NQ] O read out by the four warps
  uint64_t* drain = bars + 28;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 4);
  int* s_status = reinterpret_cast<int*>(smem + S::kOffMisc + 8);
  volatile int* met = reinterpret_cast<volatile int*>(smem + S::kOffMisc + 12);   // V held an element that is not finite
  const int warp = warp_id(), lane = lane_id();

  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    *met = 0;
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int x = 0; x < NQ; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_full[x], 1);
      mbar_init(&o_free[x], 4);
    }
    mbar_init(drain, 1);
    fence_mbarrier_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  List list;
  if (!build_list<ROWS>(cu, B, T_max, max_len, nh, classes, err, s_status, smem + S::kOffList, list)) return;
  if (item_of_round(0, list.total) < 0) return;    // the whole CTA; nothing allocated yet
  if (warp == 1) {
    tmem_alloc(tmem_slot, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // key tiles of query tile x of an item (0: the tile has no query), and of the item
  auto tiles_of = [](const CausalItem& it, int x) {
    const int q = it.q0 + x * kT;
    return q < it.len ? q / kT + 1 : 0;
  };
  auto tiles = [&](const CausalItem& it) {
    int n = tiles_of(it, 0);
    if constexpr (NQ == 2) n = max(n, tiles_of(it, 1));
    return n;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      uint32_t idx = 0;                            // ring tiles issued
      uint32_t nq[2] = {0, 0};
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
      for (int r = 0; ok; ++r) {
        const int g = item_of_round(r, list.total);
        if (g < 0) break;
        const CausalItem it = item_at<ROWS>(list, g);
        const int kv_col = it.h / group * D;
        const int n = tiles(it);
        auto load_q = [&](int x) -> bool {
          if (!tiles_of(it, x)) return true;
          if (!mbar_wait_bounded(&q_empty[x], (nq[x] & 1u) ^ 1u, abort_flag)) return false;
          mbar_arrive_expect_tx(&q_full[x], S::kTileBytes);
#pragma unroll
          for (int c = 0; c < HB; ++c)
            tma_load_2d(sQ + x * S::kTileBytes + c * kBox, &tq, &q_full[x], q_x + it.h * D + 64 * c,
                        it.c0 + it.q0 + x * kT);
          ++nq[x];
          return true;
        };
        // Q_0 K_0 before Q_1: the first scores of query tile 0 are issued before the last ones of
        // the previous item's query tile 1, which Q_1 waits for
        ok = load_q(0) && load(&tk, k_x + kv_col, it.c0);
        if constexpr (NQ == 2) ok = ok && load_q(1);
        ok = ok && load(&tv, v_x + kv_col, it.c0);
        for (int j = 1; j < n && ok; ++j)
          ok = load(&tk, k_x + kv_col, it.c0 + j * kT) && load(&tv, v_x + kv_col, it.c0 + j * kT);
      }
      if (!ok) {
        set_device_error(err, RPP_DERR_TIMEOUT);
        *abort_flag = 1;
      }
      // what is in flight lands before the CTA can exit: the last load of each buffer
      for (uint32_t i = idx > S::kSlots ? idx - S::kSlots : 0; i < idx; ++i)
        mbar_wait_bounded(&full[i % S::kSlots], (i / S::kSlots) & 1u, nullptr);
      for (int x = 0; x < NQ; ++x)
        if (nq[x]) mbar_wait_bounded(&q_full[x], (nq[x] - 1) & 1u, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr int fmt = attn::Fmt<T>::v;
      constexpr uint32_t IDESC_S = idesc_f16(fmt, kT, kT);
      constexpr uint32_t IDESC_O = idesc_f16(fmt, kT, D) | (1u << 16);   // B (= V) N-major
      // V: N-major, 64 columns a box (the second box kBox further), 8 keys 1024 bytes apart
      constexpr uint64_t kVLead = D == 128 ? (static_cast<uint64_t>(kBox >> 4) << 16) - (1ull << 16) : 0ull;
      uint32_t nq[2] = {0, 0}, np[2] = {0, 0}, no[2] = {0, 0};
      bool ok = true;
      // S(j) of tile x; `base`: ring index of the item's K_0
      auto issue_s = [&](const CausalItem& it, int x, int j, uint32_t base) -> bool {
        const uint32_t i = base + 2u * j, s = i % S::kSlots;
        if (j == 0 && !mbar_wait_bounded(&q_full[x], nq[x] & 1u, abort_flag)) return false;
        if (!mbar_wait_bounded(&full[s], (i / S::kSlots) & 1u, abort_flag)) return false;
        tc_fence_after();
        const uint32_t qa = smem_u32(sQ + x * S::kTileBytes), ka = smem_u32(ring + s * S::kTileBytes);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma_f16(tmem + 128u * x, sw128_kmajor_desc(qa + (k >> 2) * kBox) + 2u * (k & 3),
                     sw128_kmajor_desc(ka + (k >> 2) * kBox) + 2u * (k & 3), IDESC_S, k ? 1u : 0u);
        tc_commit(&s_full[x]);
        const bool last_user = x == NQ - 1 || tiles_of(it, NQ - 1) <= j;
        if (last_user) tc_commit(&empty[s]);
        if (j == tiles_of(it, x) - 1) {
          tc_commit(&q_empty[x]);
          ++nq[x];
        }
        return true;
      };
      auto issue_pv = [&](const CausalItem& it, int x, int j, uint32_t base) -> bool {
        const uint32_t i = base + 2u * j + 1u, s = i % S::kSlots;
        if (!mbar_wait_bounded(&p_full[x], np[x] & 1u, abort_flag)) return false;
        ++np[x];
        if (!mbar_wait_bounded(&full[s], (i / S::kSlots) & 1u, abort_flag)) return false;
        if (j == 0 && no[x] && !mbar_wait_bounded(&o_free[x], (no[x] - 1) & 1u, abort_flag)) return false;
        tc_fence_after();
        const uint64_t vd = sw128_kmajor_desc(smem_u32(ring + s * S::kTileBytes)) + kVLead;
#pragma unroll
        for (int k = 0; k < kT / 16; ++k)   // 16 keys: P columns +8, V +2048 bytes
          tc_mma_f16_tmem_a(tmem + S::kColO + 128u * x, tmem + 128u * x + 8u * k, vd + 128u * k, IDESC_O,
                            (j | k) ? 1u : 0u);
        const bool last_user = x == NQ - 1 || tiles_of(it, NQ - 1) <= j;
        if (last_user) tc_commit(&empty[s]);
        if (j == tiles_of(it, x) - 1) {
          tc_commit(&o_full[x]);
          ++no[x];
        }
        return true;
      };
      int r = 0;
      CausalItem it = item_at<ROWS>(list, item_of_round(0, list.total));
      uint32_t base = 0;
      bool ahead[2] = {false, false};              // S(0) of the item has been issued
      for (; ok;) {
        const int n = tiles(it);
        const int gn = item_of_round(r + 1, list.total);
        CausalItem nx = it;
        if (gn >= 0) nx = item_at<ROWS>(list, gn);
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
          if (ok && !ahead[x] && tiles_of(it, x)) ok = issue_s(it, x, 0, base);
          ahead[x] = false;
        }
        for (int j = 0; j < n && ok; ++j) {
#pragma unroll
          for (int x = 0; x < NQ; ++x) {
            const int nt = tiles_of(it, x);
            if (!ok || j >= nt) continue;
            ok = issue_pv(it, x, j, base);
            if (!ok) break;
            if (j + 1 < nt) {
              ok = issue_s(it, x, j + 1, base);
            } else if (gn >= 0 && tiles_of(nx, x) && j + 2 >= n) {
              // The next item's first scores.  Not while the item has more than one key tile
              // left for the other query tile: its ring tiles come first.
              ok = issue_s(nx, x, 0, base + 2u * n);
              ahead[x] = true;
            }
          }
        }
        if (!ok || gn < 0) break;
        base += 2u * n;
        it = nx;
        ++r;
      }
      if (!ok) {
        set_device_error(err, RPP_DERR_TIMEOUT);
        *abort_flag = 1;
      }
      tc_commit(drain);                            // every MMA done before tensor memory is freed
      mbar_wait_bounded(drain, 0, nullptr);
    }
  } else {
    // ------------------------------------------------------------ softmax: one thread a query row
    const int x = NQ == 2 ? (warp - 2) >> 2 : 0;
    const int quad = warp & 3;                     // tensor-memory lanes of this warp
    const int row = quad * 32 + lane;              // query of the tile, and V row of a diagonal tile
    const uint32_t t_s = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 128u * x;
    const uint32_t t_o = tmem + (static_cast<uint32_t>(quad * 32) << 16) + S::kColO + 128u * x;
    const uint64_t sc2 = f2_pack(scale_log2, scale_log2);
    uint32_t ns = 0, no = 0, base = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      const int w = mbar_wait_bounded(bar, parity, abort_flag) ? 1 : 0;
      return __all_sync(0xffffffffu, w) != 0;
    };
    for (int r = 0; ok; ++r) {
      const int g = item_of_round(r, list.total);
      if (g < 0) break;
      const CausalItem it = item_at<ROWS>(list, g);
      const int nt = tiles_of(it, x);
      const int q0 = it.q0 + x * kT;
      float m = neg_inf(), l = 0.f;
      for (int j = 0; j < nt; ++j) {
        if (!wait(&s_full[x], ns & 1u)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t v[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(t_s + 32 * c, v + 32 * c);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait_tied32(v + 32 * c);
        const bool diag = j == nt - 1;
        if (diag) {
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (e > row) v[e] = 0xff800000u;
        }
        float pm[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) pm[t] = fmaxf(__uint_as_float(v[t]), __uint_as_float(v[t + 4]));
#pragma unroll
        for (int e = 8; e < 128; e += 8)
#pragma unroll
          for (int t = 0; t < 4; ++t)
            pm[t] = fmaxf(fmaxf(pm[t], __uint_as_float(v[e + t])), __uint_as_float(v[e + t + 4]));
        const float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])) * scale_log2;
        // The maximum moves lazily; O may be touched because s_full came after the last PV.
        // The accesses to tensor memory are the whole warp's (factor 1 for the rows that stay).
        const bool move = mx > m + 8.0f;
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
        const float nm = m == neg_inf() ? 0.f : -m;
        const uint64_t nm2 = f2_pack(nm, nm);
        uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int a = 64 * c + 2 * e;
            const uint64_t x2 = f2_fma(f2_pack(__uint_as_float(v[a]), __uint_as_float(v[a + 1])), sc2, nm2);
            const float p0 = ex2_approx(f2_lo(x2)), p1 = ex2_approx(f2_hi(x2));
            sum2[e & 1] = f2_add(sum2[e & 1], f2_pack(p0, p1));
            v[32 * c + e] = pack2<T>(p0, p1);
          }
          tmem_st_32x32b_x32(t_s + 32 * c, v + 32 * c);
        }
        l += (f2_lo(sum2[0]) + f2_hi(sum2[0])) + (f2_lo(sum2[1]) + f2_hi(sum2[1]));
        if (diag) {
          // this thread's V row of the diagonal tile: zero past the sequence; elements that are
          // not finite are taken out, and the fact noted for good
          const uint32_t i = base + 2u * j + 1u, s = i % S::kSlots;
          if (!wait(&full[s], (i / S::kSlots) & 1u)) {
            ok = false;
            break;
          }
          const bool past = q0 + row >= it.len;
          bool hit = false;
          uint8_t* vrow = ring + s * S::kTileBytes + row * 128;
#pragma unroll
          for (int c = 0; c < HB * 8; ++c) {
            uint4* at = reinterpret_cast<uint4*>(vrow + (c >> 3) * kBox + ((c & 7) ^ (row & 7)) * 16);
            uint4 w = past ? make_uint4(0u, 0u, 0u, 0u) : *at;
            const uint32_t b0 = nonfinite2<T>(w.x), b1 = nonfinite2<T>(w.y), b2 = nonfinite2<T>(w.z),
                           b3 = nonfinite2<T>(w.w);
            const bool bad = (b0 | b1 | b2 | b3) != 0u;
            hit |= bad;
            if (past || bad) *at = make_uint4(w.x & ~b0, w.y & ~b1, w.z & ~b2, w.w & ~b3);
          }
          if (hit) *met = 1;
          fence_proxy_async_smem();
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_st_wait_tied32(v + 32 * c);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
        ++ns;
      }
      if (!ok) break;
      base += 2u * tiles(it);
      if (nt == 0) continue;
      if (!wait(&o_full[x], no & 1u)) {
        ok = false;
        break;
      }
      ++no;
      tc_fence_after();
      const float inv = 1.0f / l;
      T* orow = out + static_cast<long long>(it.c0 + q0 + row) * (static_cast<long long>(nh) * D) + it.h * D;
      // Elements taken out of a diagonal tile that this tile's queries see (its own, and the first
      // query tile's, which both query tiles read): added back from memory.  One that was not
      // taken out in time to miss the product is added twice, which changes nothing.  (The note
      // is visible here: o_full came after the p_full of both diagonal tiles.)
      const bool put_back = *met != 0;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld_32x32b_x32(t_o + 32 * c, ov);
        tmem_ld_wait_tied32(ov);
        if (put_back && q0 + row < it.len) {
          for (int k = it.q0; k <= q0 + row; ++k) {
            const T* vr = v_rows + static_cast<long long>(it.c0 + k) * kv_stride + it.h / group * D + 32 * c;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float f = to_f32(vr[e]);
              if (!isfinite(f)) ov[e] = __float_as_uint(__uint_as_float(ov[e]) + f);
            }
          }
        }
        if (q0 + row < it.len) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(ov[8 * u + e]) * inv;
            *reinterpret_cast<uint4*>(orow + 32 * c + 8 * u) =
                make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[x]);
    }
    if (!ok && lane == 0) {
      set_device_error(err, RPP_DERR_TIMEOUT);
      *abort_flag = 1;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

// The tensor maps of a call, and where the columns of q, k and v start in them.
struct Maps {
  CUtensorMap q, k, v;
  int q_x = 0, k_x = 0, v_x = 0;
};

template <typename T, int D, int NQ>
cudaError_t launch(const Maps& t, const CausalArgs& a, cudaStream_t stream) {
  using S = Shape<D, NQ>;
  constexpr int ROWS = NQ * kT;
  const int classes = (a.max_len + ROWS - 1) / ROWS;
  const size_t smem = 1024 + S::kOffList + list_bytes(a.B, classes);
  static SmemLimit limit;
  const cudaError_t e = limit.raise(attention_causal_kernel<T, D, NQ>,
                                    1024 + S::kOffList + list_bytes(kMaxPrompts, kMaxCausalLen / ROWS));
  if (e != cudaSuccess) return e;
  // never more CTAs than items: ceil(len / ROWS) <= len / ROWS + 1 for each sequence
  const long long most = (static_cast<long long>(a.T_max) / ROWS + a.B) * a.nh;
  const long long room = static_cast<long long>(NQ == 2 ? 1 : 2) * num_sms();
  const int grid = static_cast<int>(most < room ? most : room);
  return launch_pdl(attention_causal_kernel<T, D, NQ>, dim3(grid), dim3(S::kThreads), smem, stream, t.q, t.k, t.v,
                    t.q_x, t.k_x, t.v_x, static_cast<const T*>(a.v), a.kv_stride, a.cu, a.B, a.T_max, a.max_len, a.nh,
                    a.nh / a.nkv, classes, static_cast<T*>(a.out), a.scale * 1.4426950408889634f, a.err);
}

template <typename T>
cudaError_t dispatch(const Maps& t, const CausalArgs& a, int nq, cudaStream_t stream) {
  if (a.d == 64) return nq == 2 ? launch<T, 64, 2>(t, a, stream) : launch<T, 64, 1>(t, a, stream);
  return nq == 2 ? launch<T, 128, 2>(t, a, stream) : launch<T, 128, 1>(t, a, stream);
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
  if (a.q_stride == a.kv_stride && end - first <= 2u * static_cast<uintptr_t>(a.q_stride)) {
    if (!make_tmap_2d(&t.q, reinterpret_cast<const void*>(first), dt, 2, a.T_max, static_cast<int>((end - first) / 2),
                      kT, 64, CU_TENSOR_MAP_SWIZZLE_128B, a.q_stride))
      return cudaErrorInvalidValue;
    t.k = t.v = t.q;
    t.q_x = static_cast<int>((q - first) / 2);
    t.k_x = static_cast<int>((k - first) / 2);
    t.v_x = static_cast<int>((v - first) / 2);
  } else if (!make_tmap_2d(&t.q, a.q, dt, 2, a.T_max, a.nh * a.d, kT, 64, CU_TENSOR_MAP_SWIZZLE_128B, a.q_stride) ||
             !make_tmap_2d(&t.k, a.k, dt, 2, a.T_max, a.nkv * a.d, kT, 64, CU_TENSOR_MAP_SWIZZLE_128B, a.kv_stride) ||
             !make_tmap_2d(&t.v, a.v, dt, 2, a.T_max, a.nkv * a.d, kT, 64, CU_TENSOR_MAP_SWIZZLE_128B, a.kv_stride)) {
    return cudaErrorInvalidValue;
  }
  const int nq = a.max_len > kT ? 2 : 1;
  return a.dtype == RPP_F16 ? dispatch<__half>(t, a, nq, stream) : dispatch<__nv_bfloat16>(t, a, nq, stream);
}

}  // namespace rpp
