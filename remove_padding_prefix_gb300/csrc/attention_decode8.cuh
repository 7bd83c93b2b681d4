// Attention of one new token per sequence over a paged cache of 8-bit codes, grouped heads, head
// size 64 or 128, int8 or e4m3 (code8.cuh), queries and outputs fp16 or bf16:
//   o[i, h] = sum_j softmax_j(scale q[i, h] . K[j]) V[j],  K[j] = kc[j] 2^(kb(j) - 127), V[j] likewise,
// kb and vb the scale bytes of j's block in kv head h / (nh / kv heads).
// Half the bytes of the 16-bit cache (attention_decode.cu), so half the time there is for everything else: the kernel is
// bound by HBM only while a key's codes cost little to turn into operands.
//
//  * Work is cut as there (decode_line.cuh), in blocks of 2 KB of K and 2 KB of V.
//  * Products are transposed: S^T = K Q^T and O^T = V^T P^T on mma.sync m16n8k16, keys (or head columns) as the 16 rows and
//    up to 8 query heads as the 8 columns, two such for 9 to 16.  The cache is then the operand whose rows a lane holds
//    whole: the order of a contraction and the order of the result's rows are free, so a lane reads 16
//    contiguous bytes of a row from global memory and those are its operand as they are, without shared memory:
//    for K the columns 16 t .. of key rows g and g + 8 (Q's fragments take the same order), for V the columns
//    16 g .. of four keys, paired across keys by byte permutations (the output's rows take that order).
//  * Codes become f16 (exact for both types), so the products are exact in fp32.  fp16 queries are taken as they are; a bf16
//    query head is multiplied by the power of two that brings its largest element to 2^14 .. 2^15 (what that leaves below
//    f16's smallest step is under 2^-38 of the largest) and its scores by the inverse.
//  * K's scale multiplies the scores in fp32.  V's multiplies the weights, p 2^(vb - E) with E the largest vb so far,
//    before they become f16 operands; E moves as the running maximum does, and 2^E multiplies the output at the end.
//  * The maximum moves only when a score passes it by more than 8 (log2 units), asked by one vote a
//    block; its reduction over the lanes runs only then.
//  * P^T comes out of the scores' registers by two 8 x 8 transposes (movmatrix).  P is split into two f16
//    parts (p and what rounding p left), as in the 16-bit kernel.
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
};

__device__ __forceinline__ uint4 ld_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_stream2(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ void mma8(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
// CTAs an SM: two while a unit has up to 8 query heads (its registers fit twice)
inline int decode8_ctas(int group) { return num_sms() * (group <= 8 ? 2 : 1); }

template <bool kI8, int D, int NT, bool kFine>
__global__ void __launch_bounds__(kLineWarps * 32, NT == 1 ? 2 : 1) attention_decode8_kernel(const Decode8Params p) {
  constexpr int KB = kBlockBytes / D;            // keys of a block: 16 or 32
  constexpr int G = KB / 16;                     // groups of 16 keys
  constexpr int KS = D / 16;                     // k16 steps of the scores, and 16-row tiles of the output
  constexpr int CW = D / 32;                     // words of V that a lane has of a key
  constexpr int SC = kFine ? 2 : 1;              // scales a lane needs of 16 keys
  constexpr float kUp = 7.f;                     // weights (and their sum) are kept 2^7 times as large, up to 2^15
  const float kNone = __int_as_float(0xff800000);
  extern __shared__ __align__(16) uint8_t smem[];
  long long* s_pre = reinterpret_cast<long long*>(smem);    // [n + 1]
  const int warp = warp_id(), lane = lane_id();
  const int g = lane >> 2, t = lane & 3;
  pdl_wait();
  pdl_trigger();
  const long long carry = line_plan<__half, D, KB>(p, s_pre);   // (zeros are the same in both types)
  if (carry < 0) return;
  const int per_seq = p.d.kv_heads * p.parts;
  const long long total = carry * per_seq;
  if (total == 0) return;
  const long long warps = share_warps(total, static_cast<long long>(gridDim.x) * kLineWarps);
  const long long w_id = static_cast<long long>(warp) * gridDim.x + blockIdx.x;
  if (w_id >= warps) return;
  const long long f0 = share_start(total, warps, w_id), f1 = share_start(total, warps, w_id + 1);

  LineCursor ld{};                  // the block to load next
  ld.start(p, s_pre, per_seq, f0);
  LineCursor cc = ld;               // the block being computed
  if (lane == 0) p.cuts[w_id] = make_int4(ld.blk > 0 ? ld.i : -1, ld.unit, ld.blk, 0);

  const int ps = p.d.page_size;
  const uint8_t* pool = static_cast<const uint8_t*>(p.pool);
  const long long head_bytes = static_cast<long long>(ps) * D;
  const long long v_off = p.d.kv_heads * head_bytes;
  const int head_scales = ps >> p.shift, v_scales = p.d.kv_heads * head_scales;
  int page[G], row[G];              // of the block to load next
  auto read_pages = [&](const LineCursor& c) {
#pragma unroll
    for (int s = 0; s < G; ++s) {
      const int key = c.blk * KB + 16 * s;
      page[s] = 0;
      row[s] = 0;
      if (key < c.len) {
        const int at = key / ps;
        page[s] = __ldg(c.row + at);
        row[s] = key - at * ps;
      }
    }
  };
  uint32_t kr[16], vr[16];          // the block's codes: this lane's part
  int kb[G][SC], vb[G][SC];         // and scale bytes (keys g, g + 8 of 16)
  auto head_of = [&](const LineCursor& c, int s) {
    if (page[s] < 0 || page[s] >= p.d.pages) {
      if (lane == 0) set_device_error(p.err, RPP_DERR_PAGE);
      page[s] = 0;
    }
    return static_cast<long long>(page[s]) * 2 * p.d.kv_heads + c.unit / p.parts;
  };
  auto load_k = [&](const LineCursor& c) {
#pragma unroll
    for (int s = 0; s < G; ++s) {
      const long long head = head_of(c, s);
      const uint8_t* src = pool + head * head_bytes + (row[s] + g) * D + t * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          const uint4 v = ld_stream(src + 8 * h * D + 64 * x);
          uint32_t* to = kr + ((s * 2 + h) * (D / 64) + x) * 4;
          to[0] = v.x;
          to[1] = v.y;
          to[2] = v.z;
          to[3] = v.w;
        }
      const uint8_t* sc = p.scales + head * head_scales;
#pragma unroll
      for (int h = 0; h < SC; ++h) kb[s][h] = __ldg(sc + ((row[s] + (kFine ? g + 8 * h : 0)) >> p.shift));
    }
  };
  auto load_v = [&](const LineCursor& c) {
#pragma unroll
    for (int s = 0; s < G; ++s) {
      const long long head = head_of(c, s);
      const uint8_t* src = pool + head * head_bytes + v_off + (row[s] + 2 * t) * D + g * (D / 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) {              // keys 2t, 2t + 1, 2t + 8, 2t + 9
        const uint8_t* a = src + ((j & 1) + 8 * (j >> 1)) * D;
        uint32_t* to = vr + (s * 4 + j) * CW;
        if constexpr (CW == 4) {
          const uint4 v = ld_stream(a);
          to[0] = v.x;
          to[1] = v.y;
          to[2] = v.z;
          to[3] = v.w;
        } else {
          const uint2 v = ld_stream2(a);
          to[0] = v.x;
          to[1] = v.y;
        }
      }
      const uint8_t* sc = p.scales + head * head_scales + v_scales;
#pragma unroll
      for (int h = 0; h < SC; ++h) vb[s][h] = __ldg(sc + ((row[s] + (kFine ? g + 8 * h : 0)) >> p.shift));
    }
  };

  long long lf = f0 + 1;            // next block to load
  read_pages(ld);
  load_k(ld);
  load_v(ld);
  if (lf < f1) {
    ld.advance(p, s_pre, per_seq);
    read_pages(ld);
  }

  const int rows_kept = p.group < kRows ? p.group : kRows;
  uint32_t qf[NT][KS][2];
  float qs[NT][2];                  // scale (to base 2) of the scores of query heads 2t, 2t + 1
  float o[NT][KS][4];               // heads 2t, 2t + 1 of an even column, then of the odd one after it
  float m[NT][2], l[NT][2];
  int E = 0;                        // output and weights are in units of 2^(E - 127)
  bool fresh = true, whole = false;
  for (long long f = f0; f < f1; ++f) {
    const int head = cc.unit / p.parts, part = cc.unit - head * p.parts;
    const int have = min(kRows, p.group - part * kRows);
    if (fresh) {
      fresh = false;
      whole = cc.blk == 0;
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
            const uint4 v = r < have ? __ldg(reinterpret_cast<const uint4*>(q + r * D + 64 * x + 16 * t) + y)
                                     : make_uint4(0u, 0u, 0u, 0u);
            w[x * 8 + y * 4] = v.x;
            w[x * 8 + y * 4 + 1] = v.y;
            w[x * 8 + y * 4 + 2] = v.z;
            w[x * 8 + y * 4 + 3] = v.w;
          }
        float back = p.scale_log2;
        if (p.bf16) {
          uint32_t most = 0;
#pragma unroll
          for (int e = 0; e < 2 * KS; ++e) most = max(most, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
          const int field = most >> 7;           // of the largest element; 255: no number, its head's output is NaN
          const int up = field == 255 ? 0 : min(14 + 127 - field, 126);
          const float f_up = __int_as_float((127 + up) << 23);
          back *= __int_as_float((127 - up) << 23);
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
          qs[nt][c] = __shfl_sync(0xffffffffu, back, (2 * t + c) * 4);
          m[nt][c] = kNone;
          l[nt][c] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][k][e] = 0.f;
      }
      E = 0;
    }
    // ---- scores: KB keys x 8 NT heads
    float sc[G][NT][4];
#pragma unroll
    for (int s = 0; s < G; ++s) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[s][nt][e] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint2 a = decode4<kI8>(kr[(s * 2 * KS) + k]), b = decode4<kI8>(kr[(s * 2 + 1) * KS + k]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma8(sc[s][nt], a.x, b.x, a.y, b.y, qf[nt][k][0], qf[nt][k][1]);
      }
    }
#pragma unroll
    for (int s = 0; s < G; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ks = scale_of(kb[s][kFine ? h : 0]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) sc[s][nt][2 * h + c] *= ks * qs[nt][c];
      }
    int vs[G][2];                   // V's scale bytes of keys g, g + 8
#pragma unroll
    for (int s = 0; s < G; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) vs[s][h] = vb[s][kFine ? h : 0];
    const int left = cc.len - cc.blk * KB;
    if (left < KB) {                // keys past the sequence: no score, no scale, codes zero
#pragma unroll
      for (int s = 0; s < G; ++s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (16 * s + g + 8 * h < left) continue;
          vs[s][h] = 0;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) sc[s][nt][2 * h] = sc[s][nt][2 * h + 1] = kNone;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (16 * s + 2 * t + (j & 1) + 8 * (j >> 1) >= left)
#pragma unroll
            for (int w = 0; w < CW; ++w) vr[(s * 4 + j) * CW + w] = 0u;
      }
    }
    if (lf < f1) load_k(ld);
    // ---- running maximum and V's scale, lazily moved
    bool move = false;
#pragma unroll
    for (int s = 0; s < G; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        move = move || (vs[s][h] > E && vs[s][h] != 255);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) move = move || sc[s][nt][2 * h + c] > m[nt][c] + 8.f;
      }
    if (__any_sync(0xffffffffu, move)) {
      int e1 = E;
#pragma unroll
      for (int s = 0; s < G; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (vs[s][h] != 255) e1 = max(e1, vs[s][h]);
      e1 = __reduce_max_sync(0xffffffffu, e1);
      const float ae = pow2_neg(e1 - E);
      E = e1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float a[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = kNone;
#pragma unroll
          for (int s = 0; s < G; ++s) mx = fmaxf(mx, fmaxf(sc[s][nt][c], sc[s][nt][2 + c]));
#pragma unroll
          for (int x = 4; x <= 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
          a[c] = 1.f;
          if (mx > m[nt][c] + 8.f) {
            a[c] = ex2_approx(m[nt][c] - mx);
            m[nt][c] = mx;
          }
          l[nt][c] *= a[c];
          a[c] *= ae;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][k][e] *= a[e & 1];
      }
    }
    // ---- weights, and their transposes as operands
    uint32_t ph[G][NT][2], pl[G][NT][2];
#pragma unroll
    for (int s = 0; s < G; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // at most 1, as E is at least each (NaN of 255)
        const float f = vs[s][h] == 255 ? __int_as_float(0x7fffffff) : pow2_neg(E - vs[s][h]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            // a head whose scores so far are all -inf (or no numbers) keeps m = -inf: 0, not 2^(-inf + inf)
            const float n = m[nt][c] == kNone ? 0.f : kUp - m[nt][c];
            w[c] = ex2_approx(sc[s][nt][2 * h + c] + n);
            l[nt][c] += w[c];
            w[c] *= f;
          }
          const __half2 hi = __floats2half2_rn(w[0], w[1]);
          const float2 b = __half22float2(hi);
          ph[s][nt][h] = transpose8(*reinterpret_cast<const uint32_t*>(&hi));
          pl[s][nt][h] = transpose8(half2_bits(w[0] - b.x, w[1] - b.y));
        }
      }
    // ---- output
#pragma unroll
    for (int s = 0; s < G; ++s)
#pragma unroll
      for (int w = 0; w < CW; ++w) {
        const uint32_t* x = vr + s * 4 * CW + w;
        uint2 a[2], b[2];           // keys 2t, 2t + 1; keys 2t + 8, 2t + 9: columns 4w, 4w + 1, then 4w + 2, 4w + 3
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t sel = y ? 0x7362 : 0x5140;
          a[y] = decode4<kI8>(__byte_perm(x[0], x[CW], sel));
          b[y] = decode4<kI8>(__byte_perm(x[2 * CW], x[3 * CW], sel));
        }
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma8(o[nt][2 * w + y], a[y].x, a[y].y, b[y].x, b[y].y, ph[s][nt][0], ph[s][nt][1]);
            mma8(o[nt][2 * w + y], a[y].x, a[y].y, b[y].x, b[y].y, pl[s][nt][0], pl[s][nt][1]);
          }
      }
    if (lf < f1) {
      load_v(ld);
      if (++lf < f1) {
        ld.advance(p, s_pre, per_seq);
        read_pages(ld);
      }
    }
    // ---- the unit's end, or the share's
    const bool last = cc.blk == cc.nb - 1;
    if (last || f + 1 == f1) {
      const bool all = whole && last;
      const long long piece = 2 * w_id + (f - cc.blk > f0 ? 1 : 0);   // as in the 16-bit kernel
      const float unit = scale_of(E);
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
          const float inv = 1.f / sum;
#pragma unroll
          for (int e = 0; e < 2 * KS; ++e) {
            y[e] = o[nt][e >> 1][2 * (e & 1) + c] * unit;
            if (all) y[e] *= inv;
          }
          if (all) {
            uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + out0 + r * D + 2 * KS * g);
#pragma unroll
            for (int e = 0; e < KS / 4; ++e) out[e] = p.bf16 ? pack16<__nv_bfloat16>(y + 8 * e) : pack16<__half>(y + 8 * e);
          } else {
            if (g == 0) p.ml[piece * kRows + r] = make_float2(m[nt][c], sum);
            float4* acc = reinterpret_cast<float4*>(p.acc + (piece * rows_kept + r) * D + 2 * KS * g);
#pragma unroll
            for (int e = 0; e < KS / 2; ++e) acc[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          }
        }
    }
    if (f + 1 < f1) {
      const int u = cc.unit, i = cc.i;
      cc.advance(p, s_pre, per_seq);
      fresh = cc.unit != u || cc.i != i;
    }
  }
}

template <bool kI8, int D, int NT>
cudaError_t launch_codes(const Decode8Params& p, cudaStream_t stream) {
  const size_t smem = (static_cast<size_t>(p.n) + 1) * sizeof(long long);
  const int ctas = decode8_ctas(p.group);
  const cudaError_t e = launch_pdl(p.shift < 4 ? attention_decode8_kernel<kI8, D, NT, true> : attention_decode8_kernel<kI8, D, NT, false>,
                                   dim3(ctas), dim3(kLineWarps * 32), smem, stream, p);
  if (e != cudaSuccess) return e;
  return p.bf16 ? launch_join<__nv_bfloat16, D>(p, ctas * kLineWarps, stream)
                : launch_join<__half, D>(p, ctas * kLineWarps, stream);
}
template <bool kI8>
cudaError_t launch_codes(const Decode8Params& p, cudaStream_t stream) {
  if (p.group <= 8) return p.d.head_dim == 64 ? launch_codes<kI8, 64, 1>(p, stream) : launch_codes<kI8, 128, 1>(p, stream);
  return p.d.head_dim == 64 ? launch_codes<kI8, 64, 2>(p, stream) : launch_codes<kI8, 128, 2>(p, stream);
}

}  // namespace

}  // namespace rpp
