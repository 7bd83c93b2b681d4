// Attention of one new token per sequence over a paged key-value cache, grouped heads,
// head size 64 or 128, fp16 or bf16:
//   o[i, h] = sum_j softmax_j(scale q[i, h] . K[j]) V[j],  j < lens[slot i], K and V of kv
//   head h / (nh / kv heads).
// Every byte of K and V is used by nh / kv heads queries only: 4 d operations a query for
// 4 d bytes, so the kernel is bound by HBM and everything serves the loads.
//
//  * The work of a call is one line of key blocks (sequence, kv head, 8 KB of K and V
//    each 4 KB: 16 keys at d = 128, 32 at d = 64), cut into equal shares, one a WARP: no
//    length, however uneven, leaves a warp with more than one block above the mean.  The
//    lengths are on the device, so every CTA scans them in its prologue; nothing depends on
//    the host knowing them and a captured call serves any lengths.
//  * A warp keeps its own ring of three 8 KB stages (cp.async, 16 bytes a lane): no
//    barrier between warps, 128 KB in flight per SM, and the ring runs across the ends of
//    sequences.  Page numbers are read one block ahead of the copies that need them.
//  * Scores and output run on mma.sync m16n8k16, up to 16 query heads of a kv head as the
//    16 rows: a tile of tcgen05.mma is 128 rows, eight times what there is, and its
//    result would have to come back through tensor memory for each 8 KB.  The running
//    maximum, the sum and the output stay in registers in fp32; the maximum moves only when
//    it grows by more than 8 (log2 units).
//  * P is split into two 16-bit parts (p and what rounding p left), so the product with V
//    keeps about 16 bits of P: the second mma costs nothing while HBM is the bound.
//  * A (sequence, kv head) that one warp had whole is written at once.  Of one that was cut
//    each warp leaves maximum, sum and unnormalised output in the workspace, and a second
//    kernel (programmatic launch) joins the pieces in a fixed order: results do not depend on
//    timing.  It has a CTA for each query head while they are few (few units of many pieces),
//    else one for each place where the line was cut (many units of few pieces).
//
// Rows past the sequence are filled with zeros in shared memory (never read), so pool
// pages may hold anything there.  Values of the sequence that are not finite: at the end of a unit
// outputs that came out NaN in a row whose sum is a number are taken from those values again (nonfinite.cuh).
#include <type_traits>

#include "kernels.h"
#include "nonfinite.cuh"

namespace rpp {

namespace {

constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr int kStageBytes = 8192;       // K then V, 4 KB each
constexpr int kMinBlocks = 2;           // blocks a warp takes at least, while there are that many
constexpr int kRows = 16;               // query heads of one product
constexpr int kJoinThreads = 128;        // join by cuts
constexpr int kHeadThreads = 256;        // join by heads
constexpr size_t kRingBytes = static_cast<size_t>(kWarps) * kStages * kStageBytes;

struct DecodeParams {
  KvDims d;
  const void* pool;          // of the layer
  const int32_t* table;
  const int32_t* lens;
  const void* q;
  int q_stride;              // elements
  const int32_t* slots;      // null: slot i
  int n, nh;
  int group;                 // nh / kv_heads
  int parts;                 // 16-head parts of a group
  float scale_log2;
  void* out;
  long long* prefix;         // [n + 1]: key blocks before each sequence (per kv head part)
  int4* cuts;                // [warps]: where a share starts inside a unit, (sequence, unit, block in it); else -1
  float2* ml;                // [2 * warps][16]: maximum, sum
  float* acc;                // [2 * warps][min(group, 16)][d]
  int32_t* err;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (lo, hi) rounded to 16 bits in *p, and what the rounding left, rounded, in *rest
template <typename T>
__device__ __forceinline__ void split2(float lo, float hi, uint32_t* p, uint32_t* rest) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    const float2 f = __half22float2(h);
    const __half2 r = __floats2half2_rn(lo - f.x, hi - f.y);
    *p = *reinterpret_cast<const uint32_t*>(&h);
    *rest = *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo - f.x, hi - f.y);
    *p = *reinterpret_cast<const uint32_t*>(&h);
    *rest = *reinterpret_cast<const uint32_t*>(&r);
  }
}

// How the line of `total` blocks is cut over `warps` warps: the number of warps that get a
// share, where warp w's starts, and which warp has block f.
__host__ __device__ __forceinline__ long long share_warps(long long total, long long warps) {
  const long long most = (total + kMinBlocks - 1) / kMinBlocks;
  return most < warps ? most : warps;
}
__device__ __forceinline__ long long share_start(long long total, long long warps, long long w) {
  return total * w / warps;
}
__device__ __forceinline__ long long share_of(long long total, long long warps, long long f) {
  return ((f + 1) * warps + total - 1) / total - 1;
}

// the length of sequence i, 0 (and an error) where its slot or length is not one of the cache's
__device__ __forceinline__ int seq_len(const DecodeParams& p, int i, int* slot) {
  const int s = p.slots ? p.slots[i] : i;
  *slot = s;
  if (s < 0 || s >= p.d.slots) {
    set_device_error(p.err, RPP_DERR_SLOT);
    *slot = 0;
    return 0;
  }
  const int len = p.lens[s];
  if (len < 0 || static_cast<long long>(len) > static_cast<long long>(p.d.max_pages) * p.d.page_size) {
    set_device_error(p.err, RPP_DERR_LENGTH);
    return 0;
  }
  return len;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, 1) attention_decode_kernel(const DecodeParams p) {
  constexpr int KB = kStageBytes / (4 * D);      // keys of a block: 16 or 32
  constexpr int NT = KB / 8;                     // 8-key tiles of a block
  constexpr int CH = D / 8;                      // 16-byte chunks of a row
  constexpr int KS = D / 16;                     // k16 steps of the scores
  // fp16 weights (and so their sum and the output, too) are kept 2^7 times as large, up to 2^15: below the
  // smallest step of fp16, 2^-24, a weight is lost, and a long sequence has many small ones.
  constexpr float kUp = std::is_same<T, __half>::value ? 7.f : 0.f;
  extern __shared__ __align__(1024) uint8_t smem[];
  long long* s_pre = reinterpret_cast<long long*>(smem + kRingBytes);   // [n + 1]
  __shared__ int s_flag;
  __shared__ long long s_warp[kWarps];
  const int warp = warp_id(), lane = lane_id();
  pdl_wait();
  pdl_trigger();
  // one reading of the error word for the whole CTA, on its way together with the first lengths
  if (threadIdx.x == 0) s_flag = device_error_set(p.err) ? 1 : 0;
  int slot0;
  const int len0 = static_cast<int>(threadIdx.x) < p.n ? seq_len(p, threadIdx.x, &slot0) : 0;
  __syncthreads();
  if (s_flag) return;

  // ---- blocks before each sequence
  long long carry = 0;
  for (int base = 0; base < p.n; base += kWarps * 32) {
    const int i = base + threadIdx.x;
    long long v = 0;
    if (i < p.n) {
      int slot;
      v = ((base ? seq_len(p, i, &slot) : len0) + KB - 1) / KB;
    }
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    long long before = carry;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_warp[w];
      carry += s_warp[w];
    }
    if (i < p.n) s_pre[i] = before + x - v;
    __syncthreads();
  }
  if (threadIdx.x == 0) s_pre[p.n] = carry;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= p.n; i += kWarps * 32) p.prefix[i] = s_pre[i];
  const int per_seq = p.d.kv_heads * p.parts;    // units (kv head, 16-head part) of a sequence
  const long long total = carry * per_seq;
  // empty sequences: zeros
  for (int i = warp * gridDim.x + blockIdx.x; i < p.n; i += kWarps * gridDim.x) {
    if (s_pre[i + 1] != s_pre[i]) continue;
    uint4* row = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + static_cast<long long>(i) * p.nh * D);
    for (int e = lane; e < p.nh * (D / 8); e += 32) row[e] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (total == 0) return;
  const long long warps = share_warps(total, static_cast<long long>(gridDim.x) * kWarps);
  // consecutive shares go to different SMs: warp w of CTA c has share w * CTAs + c
  const long long w_id = static_cast<long long>(warp) * gridDim.x + blockIdx.x;
  if (w_id >= warps) return;
  const long long f0 = share_start(total, warps, w_id), f1 = share_start(total, warps, w_id + 1);

  // ---- where the share starts
  int i0;
  {
    int lo = 0, hi = p.n - 1;   // the last sequence that starts at or before f0 (empty ones passed over)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pre[mid] * per_seq <= f0) lo = mid;
      else hi = mid - 1;
    }
    i0 = lo;
  }
  struct Cursor {
    int i, unit, blk, nb, len;
    const int32_t* row;          // page numbers of the sequence
  };
  auto enter = [&](Cursor& c) {   // the lengths of sequence c.i
    int slot;
    c.len = seq_len(p, c.i, &slot);
    c.nb = static_cast<int>(s_pre[c.i + 1] - s_pre[c.i]);
    c.row = p.table + static_cast<long long>(slot) * p.d.max_pages;
  };
  auto advance = [&](Cursor& c) {   // to the next block of the line (only while there is one)
    if (++c.blk < c.nb) return;
    c.blk = 0;
    if (++c.unit < per_seq) return;
    c.unit = 0;
    do ++c.i;
    while (c.i < p.n - 1 && s_pre[c.i + 1] == s_pre[c.i]);
    enter(c);
  };
  Cursor ld{};
  ld.i = i0;
  enter(ld);
  {
    const long long rem = f0 - s_pre[i0] * per_seq;
    ld.unit = static_cast<int>(rem / ld.nb);
    ld.blk = static_cast<int>(rem - static_cast<long long>(ld.unit) * ld.nb);
  }
  Cursor cc = ld;                   // the block being computed
  if (lane == 0) p.cuts[w_id] = make_int4(ld.blk > 0 ? ld.i : -1, ld.unit, ld.blk, 0);

  // ---- loads: 16 bytes a lane, 8 rows-groups each of K and V
  const int ps = p.d.page_size;
  const T* pool = static_cast<const T*>(p.pool);
  const long long head_elems = static_cast<long long>(ps) * D;
  const long long v_off = static_cast<long long>(p.d.kv_heads) * head_elems;   // K to V inside a page
  const long long page_elems = 2 * v_off;
  const uint32_t ring = smem_u32(smem) + warp * (kStages * kStageBytes);
  const int lc = lane % CH, lr = lane / CH;      // chunk and row of a lane inside a row group
  constexpr int RG = 32 / CH;                    // rows of a row group
  int page[KB / 16];                             // pages of the block to load next, one per 16 keys
  auto read_pages = [&](const Cursor& c) {
#pragma unroll
    for (int s = 0; s < KB / 16; ++s) {
      const int key = c.blk * KB + 16 * s;
      page[s] = key < c.len ? __ldg(c.row + key / ps) : 0;
    }
  };
  auto issue = [&](const Cursor& c, int stage) {
    const int head = c.unit / p.parts;
    const uint32_t dst = ring + stage * kStageBytes;
#pragma unroll
    for (int s = 0; s < KB / 16; ++s) {
      const int key = c.blk * KB + 16 * s;
      const bool ok = page[s] >= 0 && page[s] < p.d.pages;
      if (!ok && lane == 0) set_device_error(p.err, RPP_DERR_PAGE);
      const T* src = pool + (ok ? page[s] : 0) * page_elems + head * head_elems +
                     static_cast<long long>(key % ps) * D + lc * 8;
#pragma unroll
      for (int g = 0; g < 16 / RG; ++g) {
        const int r = g * RG + lr;               // row inside the 16 keys
        const bool in = ok && key + r < c.len;
        const uint32_t at = dst + ((16 * s + r) * CH + (lc ^ (r & 7))) * 16;
        const T* a = in ? src + r * D : pool;
        const int bytes = in ? 16 : 0;           // 0: zero fill, nothing is read
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(a), "r"(bytes) : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + kStageBytes / 2), "l"(in ? a + v_off : pool),
                     "r"(bytes)
                     : "memory");
      }
    }
  };

  long long lf = f0;                // next block to load
  read_pages(ld);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (lf < f1) {
      issue(ld, s);
      if (++lf < f1) {
        advance(ld);
        read_pages(ld);
      }
    }
    cp_async_commit();
  }

  const int g = lane >> 2, t = lane & 3;
  uint32_t qf[KS][4];
  float o[D / 8][4];
  float m[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
  const int krow = (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;   // ldmatrix row / chunk of K
  const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vch = lane >> 4;   // and of V
  const int rows_kept = p.group < kRows ? p.group : kRows;
  int stage = 0;
  bool fresh = true;                // the unit's first block in this share
  bool whole = false;               // that block is the unit's first
  for (long long f = f0; f < f1; ++f) {
    if (fresh) {
      fresh = false;
      whole = cc.blk == 0;
      const int head = cc.unit / p.parts, part = cc.unit - head * p.parts;
      const int have = min(kRows, p.group - part * kRows);
      const T* q = static_cast<const T*>(p.q) + static_cast<long long>(cc.i) * p.q_stride +
                   static_cast<long long>(head * p.group + part * kRows) * D;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = g + (e & 1) * 8, c = 16 * k + 2 * t + (e >> 1) * 8;
          qf[k][e] = r < have ? __ldg(reinterpret_cast<const uint32_t*>(q + r * D + c)) : 0u;
        }
      }
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
      m[0] = m[1] = __int_as_float(0xff800000);
      l[0] = l[1] = 0.f;
    }
    cp_async_wait<kStages - 2>();
    __syncwarp();
    {   // the stage that the last block freed
      const int ns = stage == 0 ? kStages - 1 : stage - 1;
      if (lf < f1) {
        issue(ld, ns);
        if (++lf < f1) {
          advance(ld);
          read_pages(ld);
        }
      }
      cp_async_commit();
    }
    const uint32_t sk = ring + stage * kStageBytes, sv = sk + kStageBytes / 2;
    // ---- scores: 16 heads x KB keys
    float s[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
#pragma unroll
      for (int h = 0; h < KB / 16; ++h) {
        uint32_t b[4];
        const int r = 16 * h + krow;
        ldsm4(sk + (r * CH + ((2 * k + kch) ^ (r & 7))) * 16, b);
        mma16816<T>(s[2 * h], qf[k], b[0], b[1]);
        mma16816<T>(s[2 * h + 1], qf[k], b[2], b[3]);
      }
    }
    const int left = cc.len - cc.blk * KB;
    if (left < KB) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * j + 2 * t + (e & 1) >= left) s[j][e] = __int_as_float(0xff800000);
    }
    // ---- running maximum, lazily moved
    float mx[2] = {s[0][0], s[0][2]};
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      mx[0] = fmaxf(mx[0], fmaxf(s[j][0], s[j][1]));
      mx[1] = fmaxf(mx[1], fmaxf(s[j][2], s[j][3]));
    }
#pragma unroll
    for (int x = 1; x <= 2; x <<= 1) {
      mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], x));
      mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], x));
    }
    mx[0] *= p.scale_log2;
    mx[1] *= p.scale_log2;
    const bool move0 = mx[0] > m[0] + 8.f, move1 = mx[1] > m[1] + 8.f;
    if (__any_sync(0xffffffffu, move0 || move1)) {
      const float a0 = move0 ? ex2_approx(m[0] - mx[0]) : 1.f, a1 = move1 ? ex2_approx(m[1] - mx[1]) : 1.f;
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        o[j][0] *= a0;
        o[j][1] *= a0;
        o[j][2] *= a1;
        o[j][3] *= a1;
      }
      l[0] *= a0;
      l[1] *= a1;
      if (move0) m[0] = mx[0];
      if (move1) m[1] = mx[1];
    }
    // a row whose scores so far are all -inf keeps m = -inf: its P is 0, not 2^(-inf + inf)
    const float n0 = m[0] == __int_as_float(0xff800000) ? 0.f : kUp - m[0];
    const float n1 = m[1] == __int_as_float(0xff800000) ? 0.f : kUp - m[1];
    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float p00 = ex2_approx(fmaf(s[j][0], p.scale_log2, n0)), p01 = ex2_approx(fmaf(s[j][1], p.scale_log2, n0));
      const float p10 = ex2_approx(fmaf(s[j][2], p.scale_log2, n1)), p11 = ex2_approx(fmaf(s[j][3], p.scale_log2, n1));
      l[0] += p00 + p01;
      l[1] += p10 + p11;
      split2<T>(p00, p01, &ph[j][0], &pl[j][0]);
      split2<T>(p10, p11, &ph[j][1], &pl[j][1]);
    }
    // ---- output
#pragma unroll
    for (int h = 0; h < KB / 16; ++h) {
      const uint32_t ah[4] = {ph[2 * h][0], ph[2 * h][1], ph[2 * h + 1][0], ph[2 * h + 1][1]};
      const uint32_t al[4] = {pl[2 * h][0], pl[2 * h][1], pl[2 * h + 1][0], pl[2 * h + 1][1]};
      const int r = 16 * h + vrow;
#pragma unroll
      for (int c = 0; c < CH; c += 2) {
        uint32_t b[4];
        ldsm4_t(sv + (r * CH + ((c + vch) ^ (r & 7))) * 16, b);
        mma16816<T>(o[c], ah, b[0], b[1]);
        mma16816<T>(o[c + 1], ah, b[2], b[3]);
        mma16816<T>(o[c], al, b[0], b[1]);
        mma16816<T>(o[c + 1], al, b[2], b[3]);
      }
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
    // ---- the unit's end, or the share's
    const bool last = cc.blk == cc.nb - 1;
    if (last || f + 1 == f1) {
#pragma unroll
      for (int x = 1; x <= 2; x <<= 1) {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], x);
        l[1] += __shfl_xor_sync(0xffffffffu, l[1], x);
      }
      const int head = cc.unit / p.parts, part = cc.unit - head * p.parts;
      const int have = min(kRows, p.group - part * kRows);
      // rows whose sum is a number: all their scores are, or -inf
      bool sound[2], redo = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float nan = 0.f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) nan = max3_nan(nan, o[j][2 * e], o[j][2 * e + 1]);
        sound[e] = g + 8 * e < have && l[e] > 0.f && l[e] < __int_as_float(0x7f800000);
        redo = redo || (sound[e] && nan != nan);
      }
      if (__any_sync(0xffffffffu, redo)) {
        // The unit's keys in this share once more, eight at a time (of one page), a lane with E columns: the sum of
        // V's elements that are not finite is the output of every row that is sound.  A K row that is not finite
        // has the score -inf in such a row: weight 0, and 0 * inf is NaN.
        constexpr int E = D / 32;
        const int here = static_cast<int>(f - f0 < cc.blk ? f - f0 : cc.blk) + 1;
        const int k1 = min(cc.len, (cc.blk + 1) * KB);
        float sum[E] = {};
        uint32_t got = 0;           // columns that have one
        int next = __ldg(cc.row + (cc.blk + 1 - here) * KB / ps);
#pragma unroll 1
        for (int key = (cc.blk + 1 - here) * KB; key < k1; key += 8) {
          const int pg = next;      // read while the rows before were under way
          if (key + 8 < k1) next = __ldg(cc.row + (key + 8) / ps);
          if (pg < 0 || pg >= p.d.pages) continue;
          const T* kr = pool + pg * page_elems + head * head_elems + static_cast<long long>(key % ps) * D + lane * E;
          const T* vr = kr + v_off;
          uint32_t w[8][E / 2], bad = 0, none = 0;     // none: rows of weight 0
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < E / 2; ++e)
              w[j][e] = key + j < k1 ? *reinterpret_cast<const uint32_t*>(vr + j * D + 2 * e) : 0u;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (key + j < k1 && part_nonfinite<T, D>(kr + j * D)) none |= 1u << j;
#pragma unroll
          for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int e = 0; e < E / 2; ++e) bad |= nonfinite2<T>(w[j][e]);
          if (!__any_sync(0xffffffffu, (bad & 0x80008000u) != 0)) continue;
          none = __reduce_or_sync(0xffffffffu, none);
          bool fixed = true;
#pragma unroll
          for (int e = 0; e < E; ++e) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (!((nonfinite2<T>(w[j][e / 2]) >> (16 * (e & 1) + 15)) & 1u)) continue;
              sum[e] += (none >> j) & 1u ? __int_as_float(0x7fffffff) : half_of<T>(w[j][e / 2], e & 1);
              got |= 1u << e;
            }
            fixed = fixed && sum[e] != sum[e];
          }
          if (__all_sync(0xffffffffu, fixed)) break;   // NaN in all columns stays
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          const int from = (8 * j + 2 * t) / E;        // the lane with this one's two columns, and which of its own they are
          const uint32_t theirs = __shfl_sync(0xffffffffu, got, from) >> (2 * t & (E - 1));
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = __shfl_sync(0xffffffffu, sum[c], from);
            if constexpr (E == 4) {
              const float y = __shfl_sync(0xffffffffu, sum[2 + c], from);
              if (t & 1) x = y;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (sound[e] && ((theirs >> c) & 1u)) o[j][2 * e + c] = x;
          }
        }
      }
      if (whole && last) {
        T* out = static_cast<T*>(p.out) +
                 (static_cast<long long>(cc.i) * p.nh + head * p.group + part * kRows) * D + 2 * t;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = g + 8 * e;
          if (r >= have) continue;
          const float inv = 1.f / l[e];
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            uint32_t w, rest;
            split2<T>(o[j][2 * e] * inv, o[j][2 * e + 1] * inv, &w, &rest);
            *reinterpret_cast<uint32_t*>(out + r * D + 8 * j) = w;
          }
        }
      } else {
        // slot 0: a unit that an earlier share began (or that begins with this one); slot 1: one begun inside
        const long long piece = 2 * w_id + (f - cc.blk > f0 ? 1 : 0);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = g + 8 * e;
          if (r >= have) continue;
          if (t == 0) p.ml[piece * kRows + r] = make_float2(m[e], l[e]);
          float* acc = p.acc + (piece * rows_kept + r) * D + 2 * t;
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            *reinterpret_cast<float2*>(acc + 8 * j) = make_float2(o[j][2 * e], o[j][2 * e + 1]);
        }
      }
    }
    __syncwarp();
    if (f + 1 < f1) {
      const int u = cc.unit, i = cc.i;
      advance(cc);
      fresh = cc.unit != u || cc.i != i;
    }
  }
}

// a piece's output by its factor; one that is not finite stays (the factor may have underflowed to 0)
__device__ __forceinline__ float weighted(float a, float x) { return isfinite(x) ? a * x : x; }

// One CTA for each share of the line: if its start is the first cut of a unit, the CTA joins that
// unit's pieces.  A thread has four output elements of one head and, where there are fewer of
// those than threads, one of several groups of pieces.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 12)
    attention_decode_join_cuts_kernel(const DecodeParams p, int main_warps) {
  __shared__ int s_flag;
  __shared__ float s_m[kRows];
  __shared__ float4 s_o[kJoinThreads];
  __shared__ float s_lg[kJoinThreads];
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) s_flag = device_error_set(p.err) ? 1 : 0;
  const int w = blockIdx.x;
  const int per_seq = p.d.kv_heads * p.parts;
  const long long total = p.prefix[p.n] * per_seq;
  __syncthreads();
  if (s_flag || total == 0) return;
  const long long warps = share_warps(total, main_warps);
  if (w == 0 || w >= warps) return;
  const int4 cut = p.cuts[w];
  if (cut.x < 0) return;
  const long long b0 = share_start(total, warps, w) - cut.z;       // the unit's first block
  const long long w0 = w - 1;
  if (share_start(total, warps, w0) > b0) return;                   // an earlier cut is in the unit too
  const long long nb = p.prefix[cut.x + 1] - p.prefix[cut.x];
  const int pieces = static_cast<int>(share_of(total, warps, b0 + nb - 1) - w0 + 1);
  const int head = cut.y / p.parts, part = cut.y - head * p.parts;
  const int have = min(kRows, p.group - part * kRows);
  const int kept = p.group < kRows ? p.group : kRows;
  const long long first = 2 * w0 + (b0 > share_start(total, warps, w0) ? 1 : 0);
  auto piece = [&](int k) { return k ? 2 * (w0 + k) : first; };
  const int warp = warp_id(), lane = lane_id();
  for (int r = warp; r < have; r += kJoinThreads / 32) {
    float mx = __int_as_float(0xff800000);
    for (int k = lane; k < pieces; k += 32) mx = fmaxf(mx, p.ml[piece(k) * kRows + r].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) s_m[r] = mx == __int_as_float(0xff800000) ? 0.f : mx;
  }
  __syncthreads();
  constexpr int V = D / 4;
  const int items = have * V;                                       // at most 512
  const int groups = items < kJoinThreads ? kJoinThreads / items : 1;
  for (int base = 0; base < items; base += kJoinThreads) {
    const int grp = groups > 1 ? threadIdx.x / items : 0;
    const int item = groups > 1 ? threadIdx.x - grp * items : base + threadIdx.x;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
    if (item < items && grp < groups) {
      const int r = item / V, v = item - r * V;
      const float m = s_m[r];
#pragma unroll 2
      for (int k = grp; k < pieces; k += groups) {
        const float2 ml = p.ml[piece(k) * kRows + r];
        const float4 x = reinterpret_cast<const float4*>(p.acc + (piece(k) * kept + r) * D)[v];
        const float a = ex2_approx(ml.x - m);
        l += a * ml.y;
        acc.x += weighted(a, x.x);
        acc.y += weighted(a, x.y);
        acc.z += weighted(a, x.z);
        acc.w += weighted(a, x.w);
      }
    }
    if (groups > 1) {   // the groups' sums, in their order
      s_o[threadIdx.x] = acc;
      s_lg[threadIdx.x] = l;
      __syncthreads();
      if (static_cast<int>(threadIdx.x) < items) {
        for (int q = 1; q < groups; ++q) {
          const float4 x = s_o[q * items + threadIdx.x];
          acc.x += x.x;
          acc.y += x.y;
          acc.z += x.z;
          acc.w += x.w;
          l += s_lg[q * items + threadIdx.x];
        }
      }
    }
    if (item < items && grp == 0) {
      const int r = item / V, v = item - r * V;
      T* out = static_cast<T*>(p.out) +
               (static_cast<long long>(cut.x) * p.nh + head * p.group + part * kRows + r) * D + 4 * v;
      const float inv = 1.f / l;
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = from_f32<T>((&acc.x)[e] * inv);
    }
  }
}

// One CTA for each (sequence, query head): its warps share the pieces, a lane has D / 32 elements.
template <typename T, int D>
__global__ void __launch_bounds__(kHeadThreads)
    attention_decode_join_heads_kernel(const DecodeParams p, int main_warps) {
  constexpr int W = kHeadThreads / 32, E = D / 32;
  __shared__ int s_flag;
  __shared__ float s_m[W], s_l[W];
  __shared__ float s_o[W][D];
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) s_flag = device_error_set(p.err) ? 1 : 0;
  const int i = blockIdx.x, h = blockIdx.y;
  const long long pre = p.prefix[i], nb = p.prefix[i + 1] - pre;
  const int per_seq = p.d.kv_heads * p.parts;
  const long long total = p.prefix[p.n] * per_seq;
  __syncthreads();
  if (s_flag || nb == 0) return;
  const int warp = warp_id(), lane = lane_id();
  const long long warps = share_warps(total, main_warps);
  const int head = h / p.group, in_group = h - head * p.group;
  const int part = in_group / kRows, row = in_group - part * kRows;
  const long long b0 = pre * per_seq + (static_cast<long long>(head) * p.parts + part) * nb;   // the unit's first block
  const long long w0 = share_of(total, warps, b0);
  const int pieces = static_cast<int>(share_of(total, warps, b0 + nb - 1) - w0 + 1);
  if (pieces == 1) return;                                          // written by the warp that had it
  const int kept = p.group < kRows ? p.group : kRows;
  const long long first = 2 * w0 + (b0 > share_start(total, warps, w0) ? 1 : 0);
  auto piece = [&](int k) { return k ? 2 * (w0 + k) : first; };
  float mx = __int_as_float(0xff800000);
  for (int k = threadIdx.x; k < pieces; k += kHeadThreads) mx = fmaxf(mx, p.ml[piece(k) * kRows + row].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) s_m[warp] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) mx = fmaxf(mx, s_m[w]);
  const float m = mx == __int_as_float(0xff800000) ? 0.f : mx;
  float acc[E], l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int k = warp; k < pieces; k += W) {
    const float2 ml = p.ml[piece(k) * kRows + row];
    const float* src = p.acc + (piece(k) * kept + row) * D + lane * E;
    const float a = ex2_approx(ml.x - m);
    l += a * ml.y;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] += weighted(a, src[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  if (threadIdx.x < D) {
    float x = 0.f, z = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      x += s_o[w][threadIdx.x];
      z += s_l[w];
    }
    static_cast<T*>(p.out)[(static_cast<long long>(i) * p.nh + h) * D + threadIdx.x] = from_f32<T>(x / z);
  }
}

inline size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }
inline int decode_ctas() { return num_sms(); }

template <typename T, int D>
cudaError_t launch(const DecodeParams& p, cudaStream_t stream) {
  const size_t smem = kRingBytes + (static_cast<size_t>(p.n) + 1) * sizeof(long long);
  static SmemLimit limit;
  const cudaError_t a =
      limit.raise(attention_decode_kernel<T, D>, kRingBytes + (kKvMaxList + 1) * sizeof(long long));
  if (a != cudaSuccess) return a;
  const int ctas = decode_ctas();
  const cudaError_t e = launch_pdl(attention_decode_kernel<T, D>, dim3(ctas), dim3(kWarps * 32), smem, stream, p);
  if (e != cudaSuccess) return e;
  if (static_cast<long long>(p.n) * p.nh <= 4 * ctas)
    return launch_pdl(attention_decode_join_heads_kernel<T, D>, dim3(p.n, p.nh), dim3(kHeadThreads), 0, stream, p,
                      ctas * kWarps);
  return launch_pdl(attention_decode_join_cuts_kernel<T, D>, dim3(ctas * kWarps), dim3(kJoinThreads), 0, stream, p,
                    ctas * kWarps);
}

}  // namespace

size_t attention_decode_ws_bytes(int n, int nh, int nkv, int d) {
  const size_t pieces = 2 * static_cast<size_t>(decode_ctas()) * kWarps;
  const int group = nh / nkv, kept = group < kRows ? group : kRows;
  return up256((static_cast<size_t>(n) + 1) * sizeof(long long)) + up256(pieces / 2 * sizeof(int4)) +
         up256(pieces * kRows * sizeof(float2)) +
         up256(pieces * kept * d * sizeof(float));
}

cudaError_t launch_attention_decode(const KvDims& d, const KvState& c, rpp_dtype dtype, int layer, const void* q,
                                    int q_stride, const int32_t* slots, int n, int nh, float scale, void* out,
                                    void* ws, int32_t* err, cudaStream_t stream) {
  const size_t pieces = 2 * static_cast<size_t>(decode_ctas()) * kWarps;
  DecodeParams p{};
  p.d = d;
  p.pool = static_cast<const uint8_t*>(c.pool) +
           static_cast<size_t>(layer) * d.pages * 2 * d.kv_heads * d.page_size * d.head_dim * 2;
  p.table = c.table;
  p.lens = c.lens;
  p.q = q;
  p.q_stride = q_stride;
  p.slots = slots;
  p.n = n;
  p.nh = nh;
  p.group = nh / d.kv_heads;
  p.parts = (p.group + kRows - 1) / kRows;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.out = out;
  uint8_t* at = static_cast<uint8_t*>(ws);
  p.prefix = reinterpret_cast<long long*>(at);
  at += up256((static_cast<size_t>(n) + 1) * sizeof(long long));
  p.cuts = reinterpret_cast<int4*>(at);
  at += up256(pieces / 2 * sizeof(int4));
  p.ml = reinterpret_cast<float2*>(at);
  at += up256(pieces * kRows * sizeof(float2));
  p.acc = reinterpret_cast<float*>(at);
  p.err = err;
  if (dtype == RPP_F16)
    return d.head_dim == 64 ? launch<__half, 64>(p, stream) : launch<__half, 128>(p, stream);
  return d.head_dim == 64 ? launch<__nv_bfloat16, 64>(p, stream) : launch<__nv_bfloat16, 128>(p, stream);
}

}  // namespace rpp
