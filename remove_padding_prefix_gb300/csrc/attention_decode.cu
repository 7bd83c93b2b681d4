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
//    it grows by more than 8 (log2 units).  From maxima of 2^16 on the product of score and scale is
//    rounded on its own, as the maximum's is: in an fma it is not, and from 2^29 on the two are up to 2^32 apart.
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

#include "decode_line.cuh"
#include "nonfinite.cuh"

namespace rpp {

namespace {

constexpr int kWarps = 8;
constexpr int kStages = 3;
constexpr int kStageBytes = 8192;       // K then V, 4 KB each
constexpr size_t kRingBytes = static_cast<size_t>(kWarps) * kStages * kStageBytes;

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

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, 1) attention_decode_kernel(const DecodeParams p) {
  constexpr int KB = kStageBytes / (4 * D);      // keys of a block: 16 or 32
  constexpr int NT = KB / 8;                     // 8-key tiles of a block
  constexpr int CH = D / 8;                      // 16-byte chunks of a row
  constexpr int KS = D / 16;                     // k16 steps of the scores
  // fp16 weights (and so their sum and the output, too) are kept 2^7 times as large, up to 2^15: below the
  // smallest step of fp16, 2^-24, a weight is lost, and a long sequence has many small ones.
  constexpr float kUp = std::is_same<T, __half>::value ? 7.f : 0.f;
  constexpr float kFar = 65536.f;                // a maximum this far from 0 needs rounded products
  extern __shared__ __align__(1024) uint8_t smem[];
  long long* s_pre = reinterpret_cast<long long*>(smem + kRingBytes);   // [n + 1]
  const int warp = warp_id(), lane = lane_id();
  pdl_wait();
  pdl_trigger();
  const long long carry = line_plan<T, D, KB, kWarps>(p, s_pre);
  if (carry < 0) return;
  const int per_seq = p.d.kv_heads * p.parts;    // units (kv head, 16-head part) of a sequence
  const long long total = carry * per_seq;
  if (total == 0) return;
  const long long warps = share_warps(total, static_cast<long long>(gridDim.x) * kWarps);
  // consecutive shares go to different SMs: warp w of CTA c has share w * CTAs + c
  const long long w_id = static_cast<long long>(warp) * gridDim.x + blockIdx.x;
  if (w_id >= warps) return;
  const long long f0 = share_start(total, warps, w_id), f1 = share_start(total, warps, w_id + 1);

  // ---- where the share starts
  using Cursor = LineCursor;
  auto advance = [&](Cursor& c) { c.advance(p, s_pre, per_seq); };   // (only while there is a next block)
  Cursor ld{};                      // the block to load next
  ld.start(p, s_pre, per_seq, f0);
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
      page[s] = key < c.len ? c.row[key / ps] : 0;
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
  float m[2] = {0.f, 0.f}, l[2] = {0.f, 0.f}, n[2] = {0.f, 0.f};
  const int krow = (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;   // ldmatrix row / chunk of K
  const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vch = lane >> 4;   // and of V
  const int rows_kept = p.group < kRows ? p.group : kRows;
  int stage = 0;
  bool fresh = true;                // the unit's first block in this share
  bool whole = false;               // that block is the unit's first
  bool far = false;                 // one of the maxima is: scores are multiplied on their own,
  float by = p.scale_log2;          // by 1 in the fma then
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
          qf[k][e] = r < have ? *reinterpret_cast<const uint32_t*>(q + r * D + c) : 0u;
        }
      }
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.f;
      m[0] = m[1] = __int_as_float(0xff800000);
      l[0] = l[1] = n[0] = n[1] = 0.f;
      far = false;
      by = p.scale_log2;
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
    // (rounded down, so that no weight passes 2^15)
    const bool move0 = mx[0] > __fadd_rd(m[0], 8.f), move1 = mx[1] > __fadd_rd(m[1], 8.f);
    if (__any_sync(0xffffffffu, move0 || move1 || far)) {
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
      bool away = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        // a row whose scores so far are all -inf keeps m = -inf: its P is 0, not 2^(-inf + inf)
        if (m[e] == __int_as_float(0xff800000)) continue;
        n[e] = fabsf(m[e]) < kFar ? kUp - m[e] : __fsub_rd(kUp, m[e]);
        away = away || !(fabsf(m[e]) < kFar);
      }
      far = __any_sync(0xffffffffu, away);
      by = far ? 1.f : p.scale_log2;
      if (far)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[j][e] = __fmul_rn(s[j][e], p.scale_log2);
    }
    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float p00 = ex2_approx(fmaf(s[j][0], by, n[0])), p01 = ex2_approx(fmaf(s[j][1], by, n[0]));
      const float p10 = ex2_approx(fmaf(s[j][2], by, n[1])), p11 = ex2_approx(fmaf(s[j][3], by, n[1]));
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
        int next = cc.row[(cc.blk + 1 - here) * KB / ps];
#pragma unroll 1
        for (int key = (cc.blk + 1 - here) * KB; key < k1; key += 8) {
          const int pg = next;      // read while the rows before were under way
          if (key + 8 < k1) next = cc.row[(key + 8) / ps];
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
  return launch_join<T, D>(p, ctas * kWarps, stream);
}

}  // namespace

size_t attention_decode_ws_bytes(int n, int nh, int nkv, int d) {
  return line_ws_bytes(n, nh, nkv, d, static_cast<long long>(decode_ctas()) * kWarps);
}

cudaError_t launch_attention_decode(const KvDims& d, const KvState& c, rpp_dtype dtype, int layer, const void* q,
                                    int q_stride, const int32_t* slots, int n, int nh, float scale, void* out,
                                    void* ws, int32_t* err, cudaStream_t stream) {
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
  line_ws_bind(&p, ws, static_cast<long long>(decode_ctas()) * kWarps);
  p.err = err;
  if (dtype == RPP_F16)
    return d.head_dim == 64 ? launch<__half, 64>(p, stream) : launch<__half, 128>(p, stream);
  return d.head_dim == 64 ? launch<__nv_bfloat16, 64>(p, stream) : launch<__nv_bfloat16, 128>(p, stream);
}

}  // namespace rpp
