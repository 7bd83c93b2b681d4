// Attention of one new token per sequence over a paged cache of 8-bit codes, grouped heads, head
// size 64 or 128, int8 or e4m3 (code8.cuh), queries and outputs fp16 or bf16:
//   o[i, h] = sum_j softmax_j(scale q[i, h] . K[j]) V[j],  K[j] = kc[j] 2^(kb(j) - 127), V[j] likewise,
// kb and vb the scale bytes of j's block in kv head h / (nh / kv heads).
// Half the bytes of the 16-bit cache (attention_decode.cu), so half the time there is for everything else: the kernel is
// bound by HBM only while a key's codes cost little to turn into operands.
//
//  * Work is cut as there (decode_line.cuh), in blocks of 2 KB of K and 2 KB of V.
//  * Products are transposed: S^T = K Q^T and O^T = V^T P^T on mma.sync m16n8k16, keys (or head columns) as the 16 rows and
//    up to 8 query heads as the 8 columns, two such for 9 to 16 (operands of tcgen05.mma would have to be written back to
//    shared memory after their conversion, for results that come through tensor memory).  The order of a contraction and the order of the
//    result's rows are free, so a lane's operands are 16 bytes of a row as they lie there: of K the columns 16 t .. of
//    key rows g and g + 8 (Q's fragments take the same order), of V the columns 16 g .. of four keys, paired across
//    keys by byte permutations (the output's rows take that order).
//  * A warp keeps its own ring of blocks (cp.async, 16 bytes a lane), chunks moved inside their 128-byte line so that no
//    reading meets a bank twice: 98 to 147 KB an SM on their way or in use.  Reading the cache straight into operand
//    registers, without the ring, leaves too few bytes on their way: 128 sequences of 200 to 8192 keys, d = 128, 32 heads
//    on 8, e4m3: 238 us, with the ring then 190 (182 now); with blocks brought to L2 ahead by bulk prefetches 275 and more.
//  * Codes become f16 (exact for both types), so the products are exact in fp32.  fp16 queries are taken as they are; a bf16
//    query head is multiplied by the power of two that brings its largest element to 2^7 .. 2^8 (what that leaves below
//    f16's smallest step is under 2^-31 of the largest) and its scores by the inverse.
//  * K's scale multiplies the scores in fp32.  V's multiplies the weights before they become f16 operands, p 2^(vb - E), an
//    addition to p's exponent; 2^E multiplies the output at the end.  E is a query head's own and follows its largest
//    p 2^vb: by the largest vb alone, a block that no query looks at would push those that carry the output out of f16's
//    range (bytes 45 apart: 0).
//  * At a unit's first block the largest weight, and the largest in units of 2^E, become 2^7 to 2^8.  E moves when one
//    passes f16's largest, the maximum then, or when a lane's weights of a block (2 or 4 of a head) add up to more than 2^40:
//    so asks one vote a block, and the reductions over the lanes run only then.  Both move by whole powers of two, so sums
//    and outputs are rescaled exactly.  E of its own for each head costs 0.2 to 2% where HBM is the bound, 3 to 5% with 9 to 16 heads.
//  * A score enters a weight as fma(s, c, n), n the maximum's counterpart as it is rounded.  The product in the fma is not,
//    so weights are off by what rounding the maximum lost: nothing that matters below 2^16, but 32 powers of two at
//    2^29.  From 2^16 on (and where 0 times an infinite c is NaN) the vote is for the other way, which takes a block's
//    maximum first and rounds each product as it does there.  A score is infinite where it passes fp32's largest.
//  * P^T comes out of the scores' registers by two 8 x 8 transposes (movmatrix).  P is split into two f16
//    parts (p and what rounding p left), as in the 16-bit kernel; that costs nothing in the batch above, and cost 2 us of 61
//    for 131000 keys of 16 heads, int8, d = 64 (50.5 now).
//
// Codes past the sequence may be anything: their scores are -inf, their codes zeros.
#pragma once
#include "code8.cuh"
#include "decode_line.cuh"

namespace rpp {

namespace {

struct Decode8Params : DecodeParams {
  const uint8_t* scales;     // of the layer
  int shift;                 // log2 of a block's tokens
  int bf16;                  // type of q and out
  long long page_bytes, head_bytes, v_bytes;      // in the pool: of a page, of a head in it, from K to V
  int page_scales, head_scales, v_scales;         // and among the scales
};

__device__ __forceinline__ uint4 ld_shared4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_shared2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared1(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void copy16(uint32_t to, const uint8_t* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void mma8(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same onto zero
__device__ __forceinline__ void mma8_first(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

constexpr int kBlockBytes = 2048;                            // of K, and of V
// Warps of a CTA (one an SM) and stages of a warp's ring.  Up to 8 query heads, d = 128: 12 and 3, 182 us for 128 sequences of
// 200 to 8192 keys (e4m3); 16 and 2: 185 (but 2048 sequences of 20 keys 56.2 instead of 58.3), 12 and 2: 189.  d = 64 (twice
// the keys and so the instructions for the same bytes): 16 and 2, 50.3 us for 131000 keys of 16 heads (int8); 12 and 3:
// 55.4.  More than 8 heads: registers for 8 warps at d = 128 (3 stages 31.3 us, 4: 32.0, 2: 31.4 for 48 sequences of
// 1000 to 6000 keys, 32 heads on 2), 12 and 3 at d = 64 (192 sequences 61 us, 2 stages 70, 8 warps 80).
template <int D, int NT> struct Shape8 {
  static constexpr int kWarps = NT == 1 ? (D == 128 ? 12 : 16) : (D == 128 ? 8 : 12);
  static constexpr int kStages = NT == 1 && D == 64 ? 2 : 3;
};
constexpr size_t kScaleBytes = 256;                          // of a stage: K's and V's of up to 32 keys, 4 bytes each
template <int D, int NT> constexpr size_t ring8_bytes() {
  return Shape8<D, NT>::kWarps * Shape8<D, NT>::kStages * (2 * kBlockBytes + kScaleBytes);
}
inline int decode8_cta_warps(int group, int d) {
  if (group <= 8) return d == 128 ? Shape8<128, 1>::kWarps : Shape8<64, 1>::kWarps;
  return d == 128 ? Shape8<128, 2>::kWarps : Shape8<64, 2>::kWarps;
}
inline int decode8_warps(int group, int d) { return num_sms() * decode8_cta_warps(group, d); }

template <bool kI8, int D, int NT>
__global__ void __launch_bounds__(Shape8<D, NT>::kWarps * 32, 1) attention_decode8_kernel(const Decode8Params p) {
  constexpr int W = Shape8<D, NT>::kWarps, kStages = Shape8<D, NT>::kStages;
  constexpr int KB = kBlockBytes / D;            // keys of a block: 16 or 32
  constexpr int G = KB / 16;                     // groups of 16 keys
  constexpr int KS = D / 16;                     // k16 steps of the scores, and 16-row tiles of the output
  constexpr int CW = D / 32;                     // words of V that a lane has of a key
  constexpr int CH = D / 16, RG = 32 / CH;       // 16-byte chunks of a row, rows that the lanes copy at once
  constexpr float kUp = 7.f;                     // weights (and their sum) are kept 2^7 times as large;
  constexpr float kMost = 0x1p40f;               // where a lane's of a block add up to more, the maximum moves
  constexpr float kFar = 65536.f;                // a maximum this far from 0 needs rounded products
  constexpr int kTop = 0x477fe000;               // 65504.f: where a weight in units of 2^E is above it, E moves
  constexpr int kApart = 64 << 23;               // where V's scale is further above E than this, exponents may not be added blindly
  constexpr float kStart = 3.402823466e38f;
  constexpr int kNaN = 255 << 23;
  const float kNone = __int_as_float(0xff800000);
  extern __shared__ __align__(1024) uint8_t smem[];
  long long* s_pre = reinterpret_cast<long long*>(smem + ring8_bytes<D, NT>());   // [n + 1]
  const int warp = warp_id(), lane = lane_id();
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_trigger();
  const long long carry = line_plan<__half, D, KB, W>(p, s_pre);   // (zeros are the same in both types)
  if (carry < 0) return;
  const int per_seq = p.d.kv_heads * p.parts;
  const long long total = carry * per_seq;
  if (total == 0) return;
  const long long warps = share_warps(total, static_cast<long long>(gridDim.x) * W);
  const long long w_id = static_cast<long long>(warp) * gridDim.x + blockIdx.x;
  if (w_id >= warps) return;
  const long long f0 = share_start(total, warps, w_id), f1 = share_start(total, warps, w_id + 1);

  // ---- the block to load next
  LineCursor first{};
  first.start(p, s_pre, per_seq, f0);
  if (lane == 0) p.cuts[w_id] = make_int4(first.blk > 0 ? first.i : -1, first.unit, first.blk, 0);
  struct Place {
    int i, unit, len, left;         // sequence, unit, its keys, keys from the block on
  };
  Place ld{first.i, first.unit, first.len, first.len - first.blk * KB};
  Place cc = ld;                    // the block being computed
  bool whole = first.blk == 0, later = false;   // its unit begins in this share; with a block behind the share's first
  const int32_t* table = first.row;
  const int ps = p.d.page_size;
  const int lc = lane % CH, lr = lane / CH;      // chunk and row of a lane inside a row group
  const uint8_t *kp, *sp;           // of the unit to load, in page 0: this lane's chunk of K's first rows; its scale
  int at, row;                      // its next 16 keys: which of the sequence's pages, and the row in it
  int page[G], rows[G];             // of the block to load next
  auto head_of = [&](int unit) { return p.parts == 1 ? unit : unit / p.parts; };
  auto enter_unit = [&]() {
    const int head = head_of(ld.unit);
    kp = static_cast<const uint8_t*>(p.pool) + head * p.head_bytes + lr * D + lc * 16;
    sp = p.scales + static_cast<long long>(head) * p.head_scales + (lane < 16 ? 0 : p.v_scales);
    const int key = ld.len - ld.left;
    at = key / ps;
    row = key - at * ps;
  };
  // the next unit: the sequence's, or the first of the next sequence that is not empty
  auto next_unit = [&](Place& c) {
    if (++c.unit == per_seq) {
      c.unit = 0;
      do ++c.i;
      while (c.i < p.n - 1 && s_pre[c.i + 1] == s_pre[c.i]);
      int slot;
      c.len = seq_len(p, c.i, &slot);
    }
    c.left = c.len;
  };
  auto advance = [&]() {            // to the next block of the line (only while there is one)
    ld.left -= KB;
    if (ld.left > 0) return;
    const int i = ld.i;
    next_unit(ld);
    if (ld.i != i) table = p.table + static_cast<long long>(p.slots ? p.slots[ld.i] : ld.i) * p.d.max_pages;
    enter_unit();
  };
  auto read_pages = [&]() {
#pragma unroll
    for (int s = 0; s < G; ++s) {
      page[s] = 16 * s < ld.left ? table[at] : 0;    // past the sequence's end any page will do
      rows[s] = row;
      row += 16;
      if (row == ps) {
        row = 0;
        ++at;
      }
    }
  };
  // ---- loads: a warp's ring of kStages blocks, K then V, in 128-byte lines of eight 16-byte chunks.  Chunks are moved inside
  // their line so that the eight lanes that read at once meet all eight: D = 128, K by the row's parity (lanes g, g + 1
  // want the same four chunks), V by twice the row pair (lanes t want the same two); D = 64, a line is two rows, by
  // twice the line.
  const uint32_t ring = smem_u32(smem) + warp * (kStages * 2 * kBlockBytes);
  const uint32_t ring_sc = smem_u32(smem) + W * kStages * 2 * kBlockBytes + warp * (kStages * kScaleBytes);
  const uint32_t k_to = D == 128 ? lr * 128 + ((lc ^ ((lr & 1) << 2)) << 4)
                                 : (lr >> 1) * 128 + ((((lr & 1) * 4 + lc) ^ (lr & 6)) << 4);
  const uint32_t v_to = kBlockBytes + (D == 128 ? lr * 128 + ((lc ^ (lr & 2)) << 4) : k_to);
  int sc[G], sc_left;               // the scale bytes on their way: of lane & 15's key, K's below lane 16, V's from there
  uint32_t sc_to = 0;
  auto issue = [&](int stage) {
    const uint32_t to = ring + stage * (2 * kBlockBytes);
#pragma unroll
    for (int s = 0; s < G; ++s) {
      if (static_cast<unsigned>(page[s]) >= static_cast<unsigned>(p.d.pages)) {
        if (lane == 0) set_device_error(p.err, RPP_DERR_PAGE);
        page[s] = 0;
      }
      const uint8_t* k = kp + page[s] * p.page_bytes + rows[s] * D;
      const uint8_t* v = k + p.v_bytes;
#pragma unroll
      for (int i = 0; i < 16 / RG; ++i) {
        copy16(to + k_to + s * 1024 + i * 512, k + i * RG * D);
        copy16(to + (D == 128 && (i & 1) ? v_to ^ 64 : v_to) + s * 1024 + i * 512, v + i * RG * D);
      }
      sc[s] = sp[static_cast<long long>(page[s]) * p.page_scales + ((rows[s] + (lane & 15)) >> p.shift)];
    }
    sc_left = ld.left;
    sc_to = ring_sc + stage * kScaleBytes + lane * 4;
  };
  // K's as the float 2^(b - 126), V's shifted as far; 255 in either makes V's 255.  Keys past the sequence: of no effect (K's
  // is large, so that its product with any qs is above 0 and that with a score of -inf is -inf).
  auto keep_scales = [&]() {
#pragma unroll
    for (int s = 0; s < G; ++s) {
      const int other = __shfl_xor_sync(0xffffffffu, sc[s], 16);
      int x = lane < 16 ? sc[s] + 1 : other == 255 ? 255 : sc[s];
      if (16 * s + (lane & 15) >= sc_left) x = lane < 16 ? 253 : 0;
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(sc_to + s * 128), "r"(static_cast<uint32_t>(x) << 23) : "memory");
    }
  };

  long long todo = f1 - f0;         // blocks from the one being computed on
  enter_unit();
  read_pages();
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (s < todo) {
      if (s) keep_scales();
      issue(s);
      if (s + 1 < todo) {
        advance();
        read_pages();
      }
    }
    cp_async_commit();
  }
  int stage = 0;
  // this lane's operands in a stage
  const uint32_t k_at = D == 128 ? g * 128 + ((t + ((g & 1) << 2)) << 4) : (g >> 1) * 128 + ((((g & 1) * 4 + t) ^ (g & 6)) << 4);
  const uint32_t v_at = kBlockBytes + (D == 128 ? 2 * t * 128 + ((g ^ (2 * t)) << 4) : t * 128 + (((g >> 1) ^ (2 * t)) << 4) + (g & 1) * 8);

  const int rows_kept = p.group < kRows ? p.group : kRows;
  uint32_t qf[NT][KS][2];
  float qs[NT][2];                  // scale (to base 2) of the scores of query heads 2t, 2t + 1, times 1/2; where that is infinite
                                    // minus 2^-128 times it (-1 or less), where it is below 2^-126 minus 2^64 times it
  float o[NT][KS][4];               // heads 2t, 2t + 1 of an even column, then of the odd one after it
  float l[NT][2];                   // sums of the weights 2^(score + n):
  float n[NT][2];                   // kUp - maximum, a whole number; kStart before the first one, so that any score passes kMost
  bool odd = false;                 // one of this lane's qs is not in [0, 1]
  bool careful = false;             // products are rounded on their own
  int E[NT][2];                     // outputs and weights are in units of 2^(e - 127), E = e << 23, e 0 to 254
  int lim = -1;                     // the largest scale of V that weights may take without a look; -1: no block yet, so that
                                    // every unit's first block moves E and n
  bool fresh = true;
  for (; todo > 0; --todo) {
    if (fresh) {
      const int head = head_of(cc.unit), part = cc.unit - head * p.parts;
      const int have = min(kRows, p.group - part * kRows);
      fresh = odd = false;
      const uint16_t* q = static_cast<const uint16_t*>(p.q) + static_cast<long long>(cc.i) * p.q_stride +
                          static_cast<long long>(head * p.group + part * kRows) * D;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = 8 * nt + g;
        uint32_t w[2 * KS];
#pragma unroll
        for (int x = 0; x < D / 64; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint4 v = r < have ? reinterpret_cast<const uint4*>(q + r * D + 64 * x + 16 * t)[y]
                                     : make_uint4(0u, 0u, 0u, 0u);
            w[x * 8 + y * 4] = v.x;
            w[x * 8 + y * 4 + 1] = v.y;
            w[x * 8 + y * 4 + 2] = v.z;
            w[x * 8 + y * 4 + 3] = v.w;
          }
        float back = p.scale_log2 * 0.5f;
        if (p.bf16) {
          uint32_t most = 0;
#pragma unroll
          for (int e = 0; e < 2 * KS; ++e) most = max(most, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
          const int field = most >> 7;           // of the largest element; 255: no number, its head's output is NaN
          const int up = field == 255 || most == 0 ? 0 : min(7 + 127 - field, 110);   // (at 110 every bf16 is exact)
          const float f_up = __int_as_float((127 + up) << 23);
          const float by = __int_as_float((127 - up) << 23);
          const float x = back * by;
          back = x == __int_as_float(0x7f800000) ? -(back * 0x1p-64f * (by * 0x1p-64f)) : x < 0x1p-126f ? -(back * 0x1p64f * by) : x;
#pragma unroll
          for (int e = 0; e < 2 * KS; ++e)
            w[e] = half2_bits(__uint_as_float(w[e] << 16) * f_up, __uint_as_float(w[e] & 0xffff0000u) * f_up);
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          qf[nt][k][0] = w[2 * k];
          qf[nt][k][1] = w[2 * k + 1];
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float x = __shfl_sync(0xffffffffu, back, (2 * t + c) * 4);
          qs[nt][c] = x < 0.f ? x : fmaxf(x, 1.4e-45f);
          n[nt][c] = kStart;
          E[nt][c] = 0;
          odd = odd || !(qs[nt][c] >= 0.f && qs[nt][c] <= 1.f);
          l[nt][c] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][k][e] = 0.f;
      }
      lim = -1;
    }
    cp_async_wait<kStages - 2>();
    __syncwarp();
    keep_scales();                  // of the last block that was issued
    __syncwarp();
    {   // into the stage that the last block freed
      if (todo >= kStages) {
        issue(stage == 0 ? kStages - 1 : stage - 1);
        if (todo > kStages) {
          advance();
          read_pages();
        }
      }
      cp_async_commit();
    }
    const uint32_t here = ring + stage * (2 * kBlockBytes), here_sc = ring_sc + stage * kScaleBytes + g * 4;
    stage = stage + 1 == kStages ? 0 : stage + 1;
    // ---- scores: KB keys x 8 NT heads
    float sc[G][NT][4];
    float ks[G][2];                 // scales of keys g, g + 8: 2^(b - 126)
    int vs[G][2];                   // of V: b << 23
#pragma unroll
    for (int s = 0; s < G; ++s) {
      uint32_t kr[2][KS];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          const uint4 v = ld_shared4(here + (x ? k_at ^ 64 : k_at) + s * 1024 + h * 8 * D);
          kr[h][4 * x] = v.x;
          kr[h][4 * x + 1] = v.y;
          kr[h][4 * x + 2] = v.z;
          kr[h][4 * x + 3] = v.w;
        }
        ks[s][h] = __uint_as_float(ld_shared1(here_sc + s * 128 + h * 32));
        vs[s][h] = ld_shared1(here_sc + s * 128 + 64 + h * 32);
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint2 a = decode4<kI8>(kr[0][k]), b = decode4<kI8>(kr[1][k]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if (k == 0) mma8_first(sc[s][nt], a.x, b.x, a.y, b.y, qf[nt][k][0], qf[nt][k][1]);
          else mma8(sc[s][nt], a.x, b.x, a.y, b.y, qf[nt][k][0], qf[nt][k][1]);
      }
    }
    const int left = cc.left;
    if (left < KB) {                // keys past the sequence: no score
#pragma unroll
      for (int s = 0; s < G; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (16 * s + g + 8 * h >= left)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) sc[s][nt][2 * h] = sc[s][nt][2 * h + 1] = kNone;
    }
    // ---- weights
    float w[G][NT][4], sum[NT][2];  // (then in units of 2^E)
    bool slow = careful;
#pragma unroll
    for (int s = 0; s < G; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) slow = slow || vs[s][h] > lim;
    int most = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        sum[nt][c] = 0.f;
#pragma unroll
        for (int s = 0; s < G; ++s) {
          int x[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p = ex2_approx(fmaf(sc[s][nt][2 * h + c], ks[s][h] * qs[nt][c], n[nt][c]));
            sum[nt][c] += p;
            // (within range: p is below 2^41 or its sum too large, V's scale at most kApart above E)
            x[h] = __viaddmax_s32(__float_as_int(p), vs[s][h] - E[nt][c], 0);
            w[s][nt][2 * h + c] = __int_as_float(x[h]);
          }
          most = __vimax3_s32(most, x[0], x[1]);
        }
        slow = slow || !(sum[nt][c] <= kMost);         // (or NaN)
      }
    if (__any_sync(0xffffffffu, slow || most > kTop)) {
      // a maximum or E moves, or has to be looked at (or the unit has a block of NaN)
      bool bad = false;
#pragma unroll
      for (int s = 0; s < G; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h) bad = bad || vs[s][h] == kNaN;
      const float spoil = __any_sync(0xffffffffu, bad) ? __int_as_float(0x7fffffff) : 0.f;
      // the scores, one rounding each
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float f = qs[nt][c], up = 1.f, more = 1.f;
          if (odd) {                // powers of two kept for last: 0 times what would be infinite is 0
            if (f <= -1.f) more = 0x1p64f;
            if (f <= -1.f || f > 1.f) up = 0x1p64f;
            else if (f < 0.f) up = 0x1p-64f;
            f = f > 1.f ? f * 0x1p-64f : fabsf(f);
          }
#pragma unroll
          for (int s = 0; s < G; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& x = sc[s][nt][2 * h + c];
              x = __fmul_rn(__fmul_rn(x, f), ks[s][h]);
              if (odd) x = __fmul_rn(__fmul_rn(x, up), more);
            }
        }
      bool rare = odd;
      lim = 254 << 23;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float a[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = kNone;
#pragma unroll
          for (int s = 0; s < G; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) mx = fmaxf(mx, sc[s][nt][2 * h + c]);
#pragma unroll
          for (int x = 4; x <= 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
          int down = 0;             // how far the maximum moves
          if (mx + n[nt][c] > kUp + 6.f) {       // (not NaN: +inf on -inf)
            const float to = ceilf(kUp - mx);
            down = static_cast<int>(fminf(n[nt][c] - to, 512.f));
            n[nt][c] = to;
          }
          sum[nt][c] = 0.f;
          uint32_t high = 0;        // the largest weight times its scale, exponents added
#pragma unroll
          for (int s = 0; s < G; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float p = ex2_approx(__fadd_rn(sc[s][nt][2 * h + c], n[nt][c]));
              sum[nt][c] += p;
              w[s][nt][2 * h + c] = p;
              if (p != 0.f) high = max(high, __float_as_uint(p) + static_cast<uint32_t>(vs[s][h]));
            }
#pragma unroll
          for (int x = 4; x <= 16; x <<= 1) high = max(high, __shfl_xor_sync(0xffffffffu, high, x));
          l[nt][c] = fmaf(l[nt][c], pow2_neg(down), spoil);
          // the outputs' unit, by the move of the weights' or by this block: its largest is 2^7 to 2^8
          const int was = (E[nt][c] >> 23) - down, e = min(max(max(was, static_cast<int>(high >> 23) - 134), 0), 254);
          a[c] = pow2_neg(e - was);
          E[nt][c] = e << 23;
          lim = min(lim, min(E[nt][c], 190 << 23) + kApart);
#pragma unroll
          for (int s = 0; s < G; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int x = __viaddmax_s32(__float_as_int(w[s][nt][2 * h + c]), vs[s][h] - E[nt][c], 0);
              if (w[s][nt][2 * h + c] != 0.f) w[s][nt][2 * h + c] = __int_as_float(x);
            }
          rare = rare || !(fabsf(n[nt][c]) < kFar);
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][k][e] *= a[e & 1];
      }
      careful = false;
      if (rare) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float all = l[nt][c] + sum[nt][c];
            if (all != all) n[nt][c] = kNone;    // stays NaN, and holds up the others no more: further weights are 0
            else careful = careful || qs[nt][c] < 0.f || fabsf(n[nt][c]) >= kFar;
          }
      }
    }
    // ---- and their transposes as operands
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) l[nt][c] += sum[nt][c];
    uint32_t ph[G][NT][2], pl[G][NT][2];
#pragma unroll
    for (int s = 0; s < G; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float x = w[s][nt][2 * h], y = w[s][nt][2 * h + 1];
          const __half2 hi = __floats2half2_rn(x, y);
          ph[s][nt][h] = transpose8(*reinterpret_cast<const uint32_t*>(&hi));
          const float2 b = __half22float2(hi);
          pl[s][nt][h] = transpose8(half2_bits(x - b.x, y - b.y));
        }
    // ---- output
#pragma unroll
    for (int s = 0; s < G; ++s) {
      uint32_t vr[4][CW];           // keys 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (D == 128) {
          const uint4 v = ld_shared4(here + v_at + (j & 1) * 128 + (j >> 1) * 1024);
          vr[j][0] = v.x;
          vr[j][1] = v.y;
          vr[j][2] = v.z;
          vr[j][3] = v.w;
        } else {
          const uint2 v = ld_shared2(here + (j & 1 ? v_at ^ 64 : v_at) + s * 1024 + (j >> 1) * 512);
          vr[j][0] = v.x;
          vr[j][1] = v.y;
        }
      }
      if (left < KB) {              // what is past the sequence may be NaN
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (16 * s + 2 * t + (j & 1) + 8 * (j >> 1) >= left)
#pragma unroll
            for (int w = 0; w < CW; ++w) vr[j][w] = 0u;
      }
#pragma unroll
      for (int w = 0; w < CW; ++w) {
        uint2 a[2], b[2];           // keys 2t, 2t + 1; keys 2t + 8, 2t + 9: columns 4w, 4w + 1, then 4w + 2, 4w + 3
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t sel = y ? 0x7362 : 0x5140;
          a[y] = decode4<kI8>(__byte_perm(vr[0][w], vr[1][w], sel));
          b[y] = decode4<kI8>(__byte_perm(vr[2][w], vr[3][w], sel));
        }
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma8(o[nt][2 * w + y], a[y].x, a[y].y, b[y].x, b[y].y, ph[s][nt][0], ph[s][nt][1]);
            mma8(o[nt][2 * w + y], a[y].x, a[y].y, b[y].x, b[y].y, pl[s][nt][0], pl[s][nt][1]);
          }
      }
    }
    __syncwarp();                   // the stage is read: the next issue may fill it
    // ---- the unit's end, or the share's
    const bool last = left <= KB;
    if (last || todo == 1) {
      const int head = head_of(cc.unit), part = cc.unit - head * p.parts;
      const int have = min(kRows, p.group - part * kRows);
      const bool all = whole && last;
      const long long piece = 2 * w_id + (later ? 1 : 0);   // as in the 16-bit kernel
      const long long out0 = (static_cast<long long>(cc.i) * p.nh + head * p.group + part * kRows) * D;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float sum = l[nt][c];
#pragma unroll
          for (int x = 4; x <= 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          const int r = 8 * nt + 2 * t + c;
          if (r >= have) continue;
          float y[2 * KS];          // columns 2 KS g ..
          // of a piece: by a power of two, so that the sum is 1 to 2 and no output above twice the largest value
          const int up = sum > 0.f && sum < -kNone && fabsf(n[nt][c]) < 0x1p22f ? (__float_as_int(sum) >> 23) - 127 : 0;
          const float by = all ? 1.f / sum : __int_as_float((127 - up) << 23), unit = scale_of(E[nt][c] >> 23);
#pragma unroll
          for (int e = 0; e < 2 * KS; ++e) y[e] = o[nt][e >> 1][2 * (e & 1) + c] * by * unit;
          if (all) {
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out0 + r * D + 2 * KS * g);
#pragma unroll
            for (int e = 0; e < KS / 4; ++e) out[e] = p.bf16 ? pack16<__nv_bfloat16>(y + 8 * e) : pack16<__half>(y + 8 * e);
          } else {
            if (g == 0) p.ml[piece * kRows + r] = make_float2(static_cast<float>(up) - n[nt][c], sum * by);
            float4* acc = reinterpret_cast<float4*>(p.acc + (piece * rows_kept + r) * D + 2 * KS * g);
#pragma unroll
            for (int e = 0; e < KS / 2; ++e) acc[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          }
        }
    }
    cc.left -= KB;
    if (last && todo > 1) {
      next_unit(cc);
      fresh = whole = later = true;
    }
  }
}

// ---------------------------------------------------------------- join
constexpr int kLongUnit = 8;         // pieces of a unit that are worth a CTA for each of its heads

// One (sequence, query head) joined by the CTA's W warps, which share its pieces, in a fixed order; a lane has D / 32
// elements.  One pass: a warp's maximum and sums come from the same readings, kDeep pieces on their way, the warps' meet in
// shared memory.  pre, nb: the sequence's blocks in the line of one kv head part.
template <int W, int D> struct JoinShared8 {
  float m[W], l[W];
  float o[W][D];
};
template <typename T, int D, int W>
__device__ __forceinline__ void join_head8(const DecodeParams& p, int i, int h, long long pre, long long nb, long long total,
                                           long long warps, JoinShared8<W, D>& s) {
  // with sixteen warps for long units 12 on their way (d = 64: 131000 keys of 16 heads 49.6 us, 4: 53.8) or 8 (d = 128: 30000
  // keys, 32 heads on 8, 21.6, 4: 24.1); else 4 (8 sequences of 200 to 8192: 22.8, 8: 24.2)
  constexpr int E = D / 32, kDeep = W < 16 ? 4 : D == 64 ? 12 : 8;
  const int warp = warp_id(), lane = lane_id();
  const float kNone = __int_as_float(0xff800000);
  const int head = h / p.group, in_group = h - head * p.group;
  const int part = in_group / kRows, row = in_group - part * kRows;
  const long long b0 = pre * (p.d.kv_heads * p.parts) + (static_cast<long long>(head) * p.parts + part) * nb;
  const long long w0 = share_of(total, warps, b0);
  const int pieces = static_cast<int>(share_of(total, warps, b0 + nb - 1) - w0 + 1);
  if (pieces == 1) return;                                          // written by the warp that had it
  const int kept = p.group < kRows ? p.group : kRows;
  const long long first = 2 * w0 + (b0 > share_start(total, warps, w0) ? 1 : 0);
  float m = kNone, l = 0.f, acc[E] = {};
  for (int k0 = warp; k0 < pieces; k0 += kDeep * W) {
    float2 ml[kDeep];
    float x[kDeep][E];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int k = k0 + u * W;
      ml[u] = make_float2(kNone, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) x[u][e] = 0.f;
      if (k < pieces) {
        const long long piece = k ? 2 * (w0 + k) : first;
        ml[u] = p.ml[piece * kRows + row];
        const float* src = p.acc + (piece * kept + row) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) x[u][e] = src[e];
      }
    }
    float to = m;
#pragma unroll
    for (int u = 0; u < kDeep; ++u) to = fmaxf(to, ml[u].x);
    const float ref = to == kNone ? 0.f : to;                       // (no scores so far: 2^-inf, not 2^(-inf + inf))
    const float a0 = ex2_approx(m - ref);
    m = to;
    l *= a0;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = weighted(a0, acc[e]);
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const float a = ex2_approx(ml[u].x - ref);
      l += a * ml[u].y;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += weighted(a, x[u][e]);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s.o[warp][lane * E + e] = acc[e];
  if (lane == 0) {
    s.m[warp] = m;
    s.l[warp] = l;
  }
  __syncthreads();
  float top = kNone;
#pragma unroll
  for (int w = 0; w < W; ++w) top = fmaxf(top, s.m[w]);
  const float ref = top == kNone ? 0.f : top;
  for (int c = threadIdx.x; c < D; c += W * 32) {
    float x = 0.f, z = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float a = ex2_approx(s.m[w] - ref);
      x += weighted(a, s.o[w][c]);
      z += a * s.l[w];
    }
    static_cast<T*>(p.out)[(static_cast<long long>(i) * p.nh + h) * D + c] = from_f32<T>(x / z);
  }
}

// A CTA of kThreads for each (sequence, query head).
template <typename T, int D, int kThreads>
__global__ void __launch_bounds__(kThreads)
    attention_decode8_join_heads_kernel(const DecodeParams p, int main_warps) {
  constexpr int W = kThreads / 32;
  __shared__ int s_flag;
  __shared__ JoinShared8<W, D> s;
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x == 0) s_flag = device_error_set(p.err) ? 1 : 0;
  const int i = blockIdx.x, h = blockIdx.y;
  const long long pre = p.prefix[i], nb = p.prefix[i + 1] - pre;
  const long long total = p.prefix[p.n] * (p.d.kv_heads * p.parts);
  __syncthreads();
  if (s_flag || nb == 0) return;
  join_head8<T, D, W>(p, i, h, pre, nb, total, share_warps(total, main_warps), s);
}

// The heads of all sequences whose units have about kLongUnit pieces or more, in the order of the sequences, CTA x of
// `ctas` taking every ctas-th.
template <typename T, int D>
__device__ __forceinline__ void join_long_units(const DecodeParams& p, int main_warps, int x, int ctas) {
  constexpr int W = kJoinThreads / 32;
  __shared__ JoinShared8<W, D> s;
  __shared__ int s_seq[kJoinThreads], s_count[W];
  const int warp = warp_id(), lane = lane_id();
  const long long total = p.prefix[p.n] * (p.d.kv_heads * p.parts);
  const long long warps = share_warps(total, main_warps);
  auto is_long = [&](int i) {
    return i < p.n && total > 0 && (p.prefix[i + 1] - p.prefix[i]) * warps >= kLongUnit * total;
  };
  bool any = false;
#pragma unroll 8
  for (int i = threadIdx.x; i < p.n; i += kJoinThreads) any = any || is_long(i);
  const int failed = __syncthreads_or(device_error_set(p.err));
  if (!__syncthreads_or(any) || failed) return;
  long long before = 0, next = x;    // long sequences passed; the head to take, counted over them
  for (int base = 0; base < p.n; base += kJoinThreads) {
    const int i = base + threadIdx.x;
    const bool mine = is_long(i);
    const uint32_t who = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) s_count[warp] = __popc(who);
    __syncthreads();
    int at = __popc(who & ((1u << lane) - 1u)), count = 0;
    for (int w = 0; w < W; ++w) {
      if (w < warp) at += s_count[w];
      count += s_count[w];
    }
    if (mine) s_seq[at] = i;
    __syncthreads();
    for (; next < (before + count) * p.nh; next += ctas) {
      const int seq = s_seq[next / p.nh - before], h = static_cast<int>(next % p.nh);
      const long long pre = p.prefix[seq], nb = p.prefix[seq + 1] - pre;
      join_head8<T, D, W>(p, seq, h, pre, nb, total, warps, s);
      __syncthreads();               // s is used again
    }
    before += count;
    __syncthreads();                 // s_seq and s_count are written again
  }
}

// CTAs 0 .. main_warps - 1 have a cut each, those behind them the long units.
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 8)
    attention_decode8_join_kernel(const DecodeParams p, int main_warps) {
  pdl_wait();
  pdl_trigger();
  if (static_cast<int>(blockIdx.x) < main_warps) join_cut<T, D, kLongUnit>(p, main_warps);
  else join_long_units<T, D>(p, main_warps, blockIdx.x - main_warps, gridDim.x - main_warps);
}

// By query head where units have many pieces on the average (the lengths are on the device), with more warps the more pieces;
// else by cuts, with CTAs for the heads of long units behind.  By cuts alone, with no CTAs behind, a sequence of 100000 keys
// among 600 of 20 to 200 (32 heads on 8) took 148 us, this way 94.  131000 keys of 16 heads: 50 us with sixteen warps a
// head, 65 with four, 62 by cuts; 48 sequences of 1000 to 6000, 32 heads on 2: 31 with four, 48 with sixteen, 40 by cuts.
// 128 of 200 to 8192, 32 heads on 8: 229 with sixteen, 182 by cuts.
template <typename T, int D>
cudaError_t launch_join8(const DecodeParams& p, int warps, cudaStream_t stream) {
  constexpr int kMany = 512, kSome = 128;
  const long long units = static_cast<long long>(p.n) * p.d.kv_heads * p.parts;
  const long long heads = static_cast<long long>(p.n) * p.nh;
  if (warps >= 24 * units)
    return launch_pdl(attention_decode8_join_heads_kernel<T, D, kMany>, dim3(p.n, p.nh), dim3(kMany), 0, stream, p, warps);
  if (warps >= kLongUnit * units)
    return launch_pdl(attention_decode8_join_heads_kernel<T, D, kSome>, dim3(p.n, p.nh), dim3(kSome), 0, stream, p, warps);
  const long long most = 4 * num_sms();
  return launch_pdl(attention_decode8_join_kernel<T, D>, dim3(warps + static_cast<int>(heads < most ? heads : most)),
                    dim3(kJoinThreads), 0, stream, p, warps);
}

template <bool kI8, int D, int NT>
cudaError_t launch_codes(const Decode8Params& p, cudaStream_t stream) {
  constexpr size_t kMost = ring8_bytes<D, NT>() + (kKvMaxList + 1) * sizeof(long long);
  static_assert(kMost <= 227 * 1024);
  static SmemLimit limit;
  const cudaError_t a = limit.raise(attention_decode8_kernel<kI8, D, NT>, kMost);
  if (a != cudaSuccess) return a;
  const size_t smem = ring8_bytes<D, NT>() + (static_cast<size_t>(p.n) + 1) * sizeof(long long);
  const cudaError_t e = launch_pdl(attention_decode8_kernel<kI8, D, NT>, dim3(num_sms()), dim3(Shape8<D, NT>::kWarps * 32), smem,
                                   stream, p);
  if (e != cudaSuccess) return e;
  return p.bf16 ? launch_join8<__nv_bfloat16, D>(p, decode8_warps(p.group, D), stream)
                : launch_join8<__half, D>(p, decode8_warps(p.group, D), stream);
}
template <bool kI8>
cudaError_t launch_codes(const Decode8Params& p, cudaStream_t stream) {
  if (p.group <= 8) return p.d.head_dim == 64 ? launch_codes<kI8, 64, 1>(p, stream) : launch_codes<kI8, 128, 1>(p, stream);
  return p.d.head_dim == 64 ? launch_codes<kI8, 64, 2>(p, stream) : launch_codes<kI8, 128, 2>(p, stream);
}

}  // namespace

}  // namespace rpp
