// Writing rows into a quantised key-value cache, and reading rows of any cache back.
//
// Write: x = code * 2^(b - 127) with one byte b for each `block` tokens of a head (code8.cuh).  With a the largest magnitude
// of a block's new rows,
//   b = the smallest byte at which a is no more than half a step past the largest code,
//       or the block's own where it has rows already and that is larger;
//   code = x * 2^(127 - b), rounded half to even; codes the block has are rounded again where b grew.
// Two bytes in and one out per value and no reuse: HBM is the floor, latency the bound (7.5 instructions a value, 1.5 a cycle
// of 4, DRAM at 41% for 24 prompts of 16181 rows: a head's rows are asked for when the head before is done).  The first
// warp of a CTA finds where 16-row tiles (or blocks, if those are longer) and sequences begin among up to 32 packed
// rows; then the warps share the tiles' heads: a warp looking on its own does that for every head again, a third of all
// instructions with 8 heads (24 prompts, 16181 rows, d = 128: 26 us, this way 22.8).  A warp takes
// one head's K or V (two of 64) of up to 16 rows (or one block, if that is longer): it holds the rows in registers, 16
// bytes a lane and row, reduces the magnitudes as 16-bit pairs (NaN largest), and writes codes and scale.  So the rows are read
// once; only blocks of 32 and more tokens take their rows from L2 a second time.  fp16 rows are turned into codes
// as pairs where their scale is an f16 number, all others in fp32 (the same codes either way).
// All rows of a block that a call brings are one warp's: no atomics, and results do not depend on timing.
//
// Read: a flat copy of rows that turns codes into values on the way, one byte in and two out.
//
// Both find the sequence of a row in the list of offsets, which every CTA has in shared memory, a lane a row.
#include "code8.cuh"
#include "kv_common.cuh"

namespace rpp {

namespace {

constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kMaxTok = 32;     // packed rows that a warp looks at together (a lane each)
constexpr int kAppendCtas = 4;  // CTAs of an append that an SM holds (64 registers, which spill 24 to 84 bytes but for P = 1, D = 64, kFine)
constexpr int kReadCtas = 3;    // and of a read (80)

// The packed row t of a call: its sequence, and how far from its end (1: the last token; below 1: nobody's row).
// cu: in shared memory, or null.
__device__ __forceinline__ int row_owner(const int32_t* cu, int n, int t, long long* back) {
  if (!cu) {
    *back = 1;
    return t;
  }
  int lo = 0, hi = n - 1;         // the last i with cu[i] <= t (sequences without rows are passed over)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  *back = t < cu[lo] ? 0 : static_cast<long long>(cu[lo + 1]) - t;   // rows before cu[0] are nobody's
  return lo;
}

struct Codes {
  KvDims d;
  uint8_t* pool;              // of the layer
  uint8_t* scales;            // of the layer
  int shift;                  // log2 of a block's tokens
};

// Two 16-bit floats of a word.
template <typename T> struct Pair16;
template <> struct Pair16<__half> { using type = __half2; };
template <> struct Pair16<__nv_bfloat16> { using type = __nv_bfloat162; };
template <typename T>
__device__ __forceinline__ typename Pair16<T>::type as_pair(uint32_t w) {
  return *reinterpret_cast<const typename Pair16<T>::type*>(&w);
}
// elementwise the larger magnitude, NaN where one is; the signs mean nothing
template <typename T>
__device__ __forceinline__ uint32_t most2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (std::is_same<T, __half>::value)
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ uint32_t most8(const uint4& v) {
  return most2<T>(most2<T>(v.x, v.y), most2<T>(v.z, v.w));
}
// the larger of a word's two, without signs (bits of magnitudes, and of NaN above them, are in order)
__device__ __forceinline__ uint32_t either(uint32_t m) { return max(m & 0x7fffu, (m >> 16) & 0x7fffu); }
__device__ __forceinline__ uint32_t umax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ float of_bits(uint32_t b) {
  const unsigned short s = static_cast<unsigned short>(b);
  return to_f32(*reinterpret_cast<const T*>(&s));
}

// Whether encode8_fast may take values up to `most` at scale byte b: no saturation (int8), a scale that f16 has (fp16).
template <typename T, bool kI8>
__device__ __forceinline__ bool fast_ok(float most, int b) {
  if (b >= 254) return false;
  if (std::is_same<T, __half>::value && (b < 127 - 15 || b > 127 + 14)) return false;
  return !kI8 || most * inverse_of(b) < Code8<true>::kPast;
}
// eight values -> eight codes
template <typename T, bool kI8>
__device__ __forceinline__ uint2 encode8_fast(const uint4& w, int b) {
  uint2 r;
  if constexpr (std::is_same<T, __half>::value) {
    const unsigned short bits = static_cast<unsigned short>((15 + 127 - b) << 10);    // 2^(127 - b)
    const __half h = *reinterpret_cast<const __half*>(&bits);
    const __half2 inv = __halves2half2(h, h);
    if constexpr (kI8) {
      // 1.5 * 2^10 added: the sum's last bits are the rounded integer
      const __half2 magic = __floats2half2_rn(1536.f, 1536.f);
      __half2 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = __hfma2(as_pair<__half>((&w.x)[e]), inv, magic);
      const uint32_t* u = reinterpret_cast<const uint32_t*>(x);
      r.x = __byte_perm(u[0], u[1], 0x6420);
      r.y = __byte_perm(u[2], u[3], 0x6420);
    } else {
      uint16_t c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __half2 x = __hmul2(as_pair<__half>((&w.x)[e]), inv);
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c[e]) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
      }
      r.x = static_cast<uint32_t>(c[0]) | (static_cast<uint32_t>(c[1]) << 16);
      r.y = static_cast<uint32_t>(c[2]) | (static_cast<uint32_t>(c[3]) << 16);
    }
  } else {
    if constexpr (kI8) {
      constexpr float kMagic = 12582912.f;
      const float inv = inverse_of(b);
      float f[8];
      unpack16<T>(w, f);
      uint32_t u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = __float_as_uint(fmaf(f[e], inv, kMagic));
      r.x = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
      r.y = __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410);
    } else {
      const unsigned short bits = static_cast<unsigned short>((254 - b) << 7);          // 2^(127 - b)
      const __nv_bfloat16 h = *reinterpret_cast<const __nv_bfloat16*>(&bits);
      const __nv_bfloat162 inv = __halves2bfloat162(h, h);
      float2 f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = __bfloat1622float2(__hmul2(as_pair<__nv_bfloat16>((&w.x)[e]), inv));
      r = make_uint2(encode4<false>(f[0].x, f[0].y, f[1].x, f[1].y), encode4<false>(f[2].x, f[2].y, f[3].x, f[3].y));
    }
  }
  return r;
}
// (zeros where b is 255)
template <typename T, bool kI8>
__device__ __forceinline__ uint2 encode8_any(uint4 w, int b) {
  if (b == 255) return make_uint2(0u, 0u);
  const float inv = inverse_of(b);
  float f[8];
  unpack16<T>(w, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] *= inv;
  return make_uint2(encode4<kI8>(f[0], f[1], f[2], f[3]), encode4<kI8>(f[4], f[5], f[6], f[7]));
}

// what one warp writes for a head: rows of one 16 (or one longer block) of a page
struct Job {
  int page, at, rows;         // `rows` rows from row `at` of the page
  int t;                      // the first's packed row
  int has;                    // rows that its block has before it
};

// kFine: blocks of fewer than 16 tokens.  P: heads that a warp takes together, side by side in a row.  blockIdx.x: up to 32
// packed rows (`tok`), grid-strided; blockIdx.y: spans of `span` times P of the heads of K, then V.  The first warp
// finds where jobs begin among the rows, then the CTA's warps share jobs times heads.  Dynamic shared memory: the list's
// offsets [n + 1], the slot bitmap.
template <typename T, bool kI8, int D, int P, bool kFine>
__global__ void __launch_bounds__(kMoveThreads, kAppendCtas)
    kv8_append_kernel(Codes c, const int32_t* table, const int32_t* lens,
                      const int32_t* refs, const T* k, const T* v, int row_stride,
                      const int32_t* slots, const int32_t* cu, int n, int rows_max, int tok,
                      int span, int32_t* err) {
  constexpr int GL = D / 8;             // lanes of a head's row
  constexpr int LPR = P * GL;           // lanes of a row
  constexpr int RPS = 32 / LPR;         // rows of a step
  constexpr int S = 16 / RPS;           // steps of 16 rows
  constexpr int kTwice = GL / S;        // lanes that end up with the same row's maximum (kFine): 1 or 2
  static_assert((S == 4 || S == 8) && (kTwice == 1 || kTwice == 2), "steps and lanes of the reduction below");
  extern __shared__ int32_t s_list[];
  uint32_t* seen = reinterpret_cast<uint32_t*>(s_list + n + 1);
  __shared__ Gate gate;
  __shared__ Job s_job[kMaxTok];
  __shared__ int s_jobs;
  const int ps = c.d.page_size, heads = c.d.kv_heads;
  const int kh0 = blockIdx.y * span, khs = min(span, 2 * heads / P - kh0);   // this CTA's heads, P at a time
  pdl_wait();
  pdl_trigger();
  const int first = static_cast<int>(threadIdx.x) < n ? slots[threadIdx.x] : 0;
  int c0 = 0, c1 = 0;
  if (cu) {
    if (static_cast<int>(threadIdx.x) < n) {
      c0 = cu[threadIdx.x];
      c1 = cu[threadIdx.x + 1];
    }
    for (int i = threadIdx.x; i <= n; i += kMoveThreads) s_list[i] = i == static_cast<int>(threadIdx.x) && i < n ? c0 : cu[i];
  }
  if (!pass(slots, n, first, c.d, seen, &gate, err, cu, c0, c1)) return;
  const int32_t* offs = cu ? s_list : nullptr;
  const int T_rows = cu ? s_list[n] : n;
  if ((cu && s_list[0] < 0) || T_rows > rows_max) {
    if (threadIdx.x == 0) set_device_error(err, RPP_DERR_ROWS);
    return;
  }
  const int block = 1 << c.shift, unit = kFine || block < 16 ? 16 : block;    // rows of a job at most
  const int head_scales = ps >> c.shift;
  const long long head_bytes = static_cast<long long>(ps) * D;
  const int warp = warp_id(), lane = lane_id();
  const int lr = lane / LPR, lc = lane % LPR, lg = lane % GL, lh = lc / GL;     // lh: which of the P heads
  // the warps side by side over the heads (K's, then V's), those that are left over the jobs
  const int wide = khs >= kMoveWarps ? kMoveWarps : khs >= 4 ? 4 : khs >= 2 ? 2 : 1, first_kh = kh0 + warp % wide;
  const int chunks = (T_rows + tok - 1) / tok;
  for (int ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
    if (warp == 0) {
      // which of the rows begin a job: a sequence's first, and those at a multiple of `unit`
      Job x{};
      bool lead = false;
      const int t = ch * tok + lane;
      if (lane < tok && t < T_rows) {
        long long back;
        const int i = row_owner(offs, n, t, &back);
        const int s = slots[i], len = lens[s];
        if (!len_ok(len, c.d) || back < 1 || back > len) {
          set_device_error(err, RPP_DERR_LENGTH);
        } else {
          const int pos = static_cast<int>(len - back);
          const bool begin = !cu || t == offs[i];
          if (begin || (pos & (unit - 1)) == 0) {
            const int in_seq = static_cast<int>(static_cast<unsigned>(pos) / static_cast<unsigned>(ps));
            x.page = table[static_cast<long long>(s) * c.d.max_pages + in_seq];
            if (x.page < 0 || x.page >= c.d.pages || refs[x.page] != 1) {    // not its own page
              set_device_error(err, RPP_DERR_PAGE);
            } else {
              lead = true;
              const int room = unit - (pos & (unit - 1));
              x.at = pos - in_seq * ps;
              x.rows = back < room ? static_cast<int>(back) : room;
              x.t = t;
              x.has = begin ? pos & (block - 1) : 0;
            }
          }
        }
      }
      const uint32_t who = __ballot_sync(0xffffffffu, lead);
      if (lead) s_job[__popc(who & ((1u << lane) - 1u))] = x;
      if (lane == 0) s_jobs = __popc(who);
    }
    __syncthreads();
    for (int j = warp / wide; j < s_jobs; j += kMoveWarps / wide) {
      const Job x = s_job[j];
      const int has = x.has, o0 = x.at & (unit - 1), o1 = o0 + x.rows;   // the new rows' places among the unit's
      const int r0 = x.at - o0;                                       // the unit's place in the page
      const int b0 = o0 >> c.shift;                                   // the block that may have rows
      const long long head = static_cast<long long>(x.page) * 2 * heads + first_kh * P + lh;
      uint8_t* codes = c.pool + head * head_bytes + r0 * D;
      uint8_t* scales = c.scales + head * head_scales + (r0 >> c.shift);
      const long long row0 = static_cast<long long>(x.t + lr - o0) * row_stride + lc * 8;   // the unit's row lr
      for (int kh = first_kh; kh < kh0 + khs; kh += wide, codes += wide * P * head_bytes, scales += wide * P * head_scales) {
        const int had = has ? scales[b0] : 0;
        const T* src = (kh * P < heads ? k + kh * P * D : v + (kh * P - heads) * D) + row0;
        uint4 w[S];
        auto load = [&](int base) {
          const T* a = src + static_cast<long long>(base) * row_stride;
          if (base >= o0 && base + 16 <= o1) {      // all 16 rows
#pragma unroll
            for (int s = 0; s < S; ++s) {
              w[s] = *reinterpret_cast<const uint4*>(a);
              a += static_cast<long long>(RPS) * row_stride;
            }
            return;
          }
#pragma unroll
          for (int s = 0; s < S; ++s) {
            const int o = base + s * RPS + lr;
            w[s] = make_uint4(0u, 0u, 0u, 0u);
            if (o >= o0 && o < o1) w[s] = *reinterpret_cast<const uint4*>(a);
            a += static_cast<long long>(RPS) * row_stride;
          }
        };
        int b = 0;                // a scale byte: kFine, of one row for each lane; else of the block
        bool fast;                // (the same in the whole warp)
        auto store = [&](int base) {
          uint8_t* to = codes + (base + lr) * D + lg * 8;
          int bs[S];              // of the rows that the lane stores
#pragma unroll
          for (int s = 0; s < S; ++s) bs[s] = kFine ? __shfl_sync(0xffffffffu, b, lr * LPR + lh * GL + s * kTwice) : b;
          if (fast && base >= o0 && base + 16 <= o1) {
#pragma unroll
            for (int s = 0; s < S; ++s) *reinterpret_cast<uint2*>(to + s * RPS * D) = encode8_fast<T, kI8>(w[s], bs[s]);
          } else {
#pragma unroll
            for (int s = 0; s < S; ++s) {
              const int o = base + s * RPS + lr;
              if (o >= o0 && o < o1) *reinterpret_cast<uint2*>(to + s * RPS * D) = encode8_any<T, kI8>(w[s], bs[s]);
            }
          }
        };
        int lead_b;               // the scale byte of the block that may have rows
        int mine = 0;             // kFine: the lane's row
        if constexpr (kFine) {
          // The rows' maxima, each in kTwice lanes at the end: the lanes of a head's row swap half of what they have with
          // the lane GL / 2 on, then GL / 4 and so on, so the row's step is in the lane's upper bits.
          load(0);
          uint32_t z[S / 2];
#pragma unroll
          for (int s = 0; s < S / 2; ++s) z[s] = either(most8<T>(w[s])) | either(most8<T>(w[s + S / 2])) << 16;
          {   // z[s]: steps s (low) and s + S / 2 (high)
            const bool up = lg & (GL / 2);
#pragma unroll
            for (int s = 0; s < S / 2; ++s) {
              const uint32_t y = umax2(z[s], __shfl_xor_sync(0xffffffffu, z[s], GL / 2));
              z[s] = up ? y >> 16 : y & 0xffffu;
            }
          }
#pragma unroll
          for (int n2 = S / 4, bit = GL / 4; n2 > 0; n2 >>= 1, bit >>= 1) {
            const bool up = lg & bit;
#pragma unroll
            for (int s = 0; s < n2; ++s) {
              const uint32_t give = up ? z[s] : z[s + n2], keep = up ? z[s + n2] : z[s];
              z[s] = max(keep, __shfl_xor_sync(0xffffffffu, give, bit));
            }
          }
          if constexpr (kTwice == 2) z[0] = max(z[0], __shfl_xor_sync(0xffffffffu, z[0], 1));
          mine = lg / kTwice * RPS + lr;
          // the rows of a block: a row's bits are lr's, then the lane's upper ones
#pragma unroll
          for (int q = 1; q < 8; q <<= 1)
            if (q < block) z[0] = max(z[0], __shfl_xor_sync(0xffffffffu, z[0], q < RPS ? q * LPR : q / RPS * kTwice));
          const float most = of_bits<T>(z[0]);
          b = scale_byte<kI8>(most);
          const bool shares = has && (mine >> c.shift) == b0;
          if (shares) b = max(b, had);
          fast = __all_sync(0xffffffffu, mine < o0 || mine >= o1 || fast_ok<T, kI8>(most, b));
          lead_b = shares ? b : 0;
          if (has) {
#pragma unroll
            for (int q = 1; q < 32; q <<= 1)     // all lanes of the head
              if (q < GL || q >= LPR) lead_b = max(lead_b, __shfl_xor_sync(0xffffffffu, lead_b, q));
          }
        } else {
          const int first16 = o0 & ~15, last16 = (o1 - 1) & ~15;
          uint32_t m = 0;
          for (int base = first16; base <= last16; base += 16) {
            load(base);
#pragma unroll
            for (int s = 0; s < S; ++s) m = most2<T>(m, most8<T>(w[s]));
          }
          m = either(m);
          if constexpr (P == 1) {
            m = __reduce_max_sync(0xffffffffu, m);
          } else {
#pragma unroll
            for (int q = 1; q < 32; q <<= 1)     // all lanes of the head
              if (q < GL || q >= LPR) m = max(m, __shfl_xor_sync(0xffffffffu, m, q));
          }
          const float most = of_bits<T>(m);
          b = lead_b = max(scale_byte<kI8>(most), had);
          fast = __all_sync(0xffffffffu, fast_ok<T, kI8>(most, lead_b));
        }
        if (has && __any_sync(0xffffffffu, lead_b > had && lead_b != 255)) {       // (a byte of 255 stays for the block's life)
#pragma unroll
          for (int e = 0; e < P; ++e) {          // one of the heads after the other
            const int now = __shfl_sync(0xffffffffu, lead_b, e * GL), was = __shfl_sync(0xffffffffu, had, e * GL);
            if (now <= was || now == 255) continue;
            const float f = pow2_neg(now - was);
            uint4* old = reinterpret_cast<uint4*>(codes + (e - lh) * head_bytes + (b0 << c.shift) * D);
            const int vecs = has * (D / 16);
            uint4 next = lane < vecs ? old[lane] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
            for (int i = lane; i < vecs; i += 32) {
              uint4 z = next;
              if (i + 32 < vecs) next = old[i + 32];
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const float4 y = decode4f<kI8>((&z.x)[h]);
                (&z.x)[h] = encode4<kI8>(y.x * f, y.y * f, y.z * f, y.w * f);
              }
              old[i] = z;
            }
          }
        }
        if constexpr (kFine) {
          store(0);
          if (lg % kTwice == 0 && mine >= o0 && mine < o1 && mine == max(o0, mine & ~(block - 1)))
            scales[mine >> c.shift] = static_cast<uint8_t>(b);
        } else {
          const int first16 = o0 & ~15, last16 = (o1 - 1) & ~15;
          for (int base = last16; base >= first16; base -= 16) {    // the last 16 are in hand
            if (base != last16) load(base);
            store(base);
          }
          if (lr == 0 && lg == 0) scales[b0] = static_cast<uint8_t>(lead_b);
        }
      }
    }
    __syncthreads();   // s_job is rewritten for the next rows
  }
}

// ---------------------------------------------------------------- read
__device__ __forceinline__ uint32_t pack_sat(float lo, float hi, __half) {
  uint32_t r;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_sat(float lo, float hi, __nv_bfloat16) {
  uint32_t r;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

enum { kPlain16 = 0, kInt8 = 1, kE4m3 = 2 };

// Rows of K and V of the sequences in `slots` to packed rows.  Items: up to 32 packed rows (`tok`), a warp each.  A lane
// takes eight values at a time, kDeep in flight; a row of fewer vectors than a warp has lanes shares the
// warp with the next rows.  vshift: log2 of a head's vectors, -1 if they are not a power of two up to 32.
// Dynamic shared memory: the list's offsets [n + 1].
template <typename TO, int kCode>
__global__ void __launch_bounds__(kMoveThreads, kReadCtas)
    kv_read_kernel(Codes c, const int32_t* table, const int32_t* lens,
                   const int32_t* slots, const int32_t* starts, const int32_t* cu,
                   int n, int rows_max, int tok, int vshift, TO* __restrict__ k, TO* __restrict__ v, int row_stride,
                   int32_t* err) {
  using Vec8 = typename std::conditional<kCode == kPlain16, uint4, uint2>::type;     // eight values in the pool
  constexpr int kDeep = kCode == kPlain16 ? 4 : 8;
  extern __shared__ int32_t s_list[];
  __shared__ int s_flag;
  pdl_wait();
  pdl_trigger();
  int bad = 0;
  for (int i = threadIdx.x; i < n; i += kMoveThreads) {
    const int s = slots[i];
    if (s < 0 || s >= c.d.slots) bad |= 2;
    if (cu) {
      const int a = cu[i], e = cu[i + 1];
      if (e < a) bad |= 1;
      s_list[i] = a;
      if (i == n - 1) s_list[n] = e;
    }
  }
  if (quit(err, &s_flag)) return;
  const int wrong = __syncthreads_or(bad & 2), back_step = __syncthreads_or(bad & 1);
  const int32_t* offs = cu ? s_list : nullptr;
  const int T_rows = cu ? s_list[n] : n;
  if (wrong || back_step || (cu && s_list[0] < 0) || T_rows > rows_max) {
    if (threadIdx.x == 0) set_device_error(err, wrong ? RPP_DERR_SLOT : back_step ? RPP_DERR_LENGTH : RPP_DERR_ROWS);
    return;
  }
  const int ps = c.d.page_size, heads = c.d.kv_heads;
  const int vpr = c.d.head_dim / 8;                 // vectors of a head's row
  const int half = heads * vpr, per = 2 * half;
  const int head_scales = ps >> c.shift;
  const Vec8* pool = reinterpret_cast<const Vec8*>(c.pool);
  const int warp = warp_id(), lane = lane_id();
  const int group = per < 32 ? 32 / per : 1;        // rows that a warp takes at once
  const int lr = per < 32 ? lane / per : 0, lc = per < 32 ? lane - lr * per : lane;
  const int chunks = (T_rows + tok - 1) / tok;
  for (int ch = blockIdx.x * kMoveWarps + warp; ch < chunks; ch += gridDim.x * kMoveWarps) {
    const int t0 = ch * tok, have = min(tok, T_rows - t0);
    int page = -1, row = 0;                         // of packed row t0 + lane
    if (lane < have) {
      const int t = t0 + lane;
      long long back;
      const int i = row_owner(offs, n, t, &back);
      const int s = slots[i], len = lens[s], from = starts ? starts[i] : 0;
      const long long pos = starts ? static_cast<long long>(from) + (cu ? t - offs[i] : 0) : len - back;
      if (!len_ok(len, c.d) || back < 1 || from < 0 || pos < 0 || pos >= len) {
        set_device_error(err, RPP_DERR_LENGTH);
      } else {
        const int q = static_cast<int>(pos);
        page = table[static_cast<long long>(s) * c.d.max_pages + q / ps];
        row = q % ps;
        if (page < 0 || page >= c.d.pages) {
          set_device_error(err, RPP_DERR_PAGE);
          page = -1;
        }
      }
    }
    for (int r0 = 0; r0 < have; r0 += group) {
      const int r = r0 + lr;
      const int p = __shfl_sync(0xffffffffu, page, r & 31), y = __shfl_sync(0xffffffffu, row, r & 31);
      if (p < 0 || r >= have || lr >= group) continue;
      const long long page_head = static_cast<long long>(p) * 2 * heads;
      const long long out_row = static_cast<long long>(t0 + r) * row_stride;
      for (int v0 = lc; v0 < per; v0 += kDeep * 32) {
        Vec8 x[kDeep];
        int b[kDeep];
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
          const int w = v0 + u * 32;
          if (w >= per || (u && per < 32)) break;
          const int kh = vshift >= 0 ? w >> vshift : w / vpr;    // K's heads, then V's
          x[u] = pool[((page_head + kh) * ps + y) * vpr + (w - kh * vpr)];
          if constexpr (kCode != kPlain16) b[u] = c.scales[(page_head + kh) * head_scales + (y >> c.shift)];
        }
#pragma unroll
        for (int u = 0; u < kDeep; ++u) {
          const int w = v0 + u * 32;
          if (w >= per || (u && per < 32)) break;
          uint4* to = reinterpret_cast<uint4*>((w < half ? k + w * 8 : v + (w - half) * 8) + out_row);
          if constexpr (kCode == kPlain16) {
            *to = x[u];
          } else {
            const float f = scale_of(b[u]);
            uint4 o;
            const float4 lo = decode4f<kCode == kInt8>(x[u].x), hi = decode4f<kCode == kInt8>(x[u].y);
            o.x = pack_sat(lo.x * f, lo.y * f, TO{});
            o.y = pack_sat(lo.z * f, lo.w * f, TO{});
            o.z = pack_sat(hi.x * f, hi.y * f, TO{});
            o.w = pack_sat(hi.z * f, hi.w * f, TO{});
            *to = o;
          }
        }
        if (per < 32) break;
      }
    }
  }
}

Codes codes_of(const KvDims& d, const KvState& s, const Kv8Scales& q, int layer) {
  const size_t heads = static_cast<size_t>(d.pages) * 2 * d.kv_heads;
  Codes c{d, static_cast<uint8_t*>(s.pool), q.scales, q.shift};
  c.pool += static_cast<size_t>(layer) * heads * d.page_size * d.head_dim;
  c.scales += static_cast<size_t>(layer) * heads * (d.page_size >> q.shift);
  return c;
}

struct AppendCall {
  Codes c;
  const KvState* s;
  const void *k, *v;
  int row_stride;
  const int32_t *slots, *cu;
  int n, rows_max;
  int32_t* err;
  cudaStream_t stream;
};

template <typename T, bool kI8, int D, int P>
cudaError_t append(const AppendCall& a) {
  const size_t smem = (static_cast<size_t>(a.n) + 1 + (a.c.d.slots + 31) / 32) * 4;
  // One wave of CTAs, with equal shares of the rows (up to 32 at a time); where there are fewer rows than that, CTAs share
  // the heads of a row, eight (a warp's each) at least.  Two waves: 26.8 us instead of 22.8 for the prompts above.
  const long long ctas = kAppendCtas * num_sms(), passes = (a.rows_max + ctas * kMaxTok - 1) / (ctas * kMaxTok);
  const int tok = static_cast<int>((a.rows_max + ctas * passes - 1) / (ctas * passes));
  const int x = blocks_for((static_cast<long long>(a.rows_max) + tok - 1) / tok, static_cast<int>(ctas));
  const int khs = 2 * a.c.d.kv_heads / P, most = (khs + kMoveWarps - 1) / kMoveWarps, room = static_cast<int>(ctas / x);
  const int parts = most < room ? most : room;
  const int span = (khs + parts - 1) / parts;
  const dim3 grid(x, (khs + span - 1) / span);
  return launch_pdl(a.c.shift < 4 ? kv8_append_kernel<T, kI8, D, P, true> : kv8_append_kernel<T, kI8, D, P, false>, grid,
                    dim3(kMoveThreads), smem, a.stream, a.c, static_cast<const int32_t*>(a.s->table),
                    static_cast<const int32_t*>(a.s->lens), static_cast<const int32_t*>(a.s->refs),
                    static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.row_stride, a.slots, a.cu, a.n, a.rows_max,
                    tok, span, a.err);
}
template <typename T, bool kI8>
cudaError_t append(const AppendCall& a) {
  if (a.c.d.head_dim == 128) return append<T, kI8, 128, 1>(a);
  // Two heads of 64 at a time, once there are rows for every CTA: 23192 rows of 16 heads with a scale a token 31.6 us, one at
  // a time 37.5; but one row of 12 heads 5.4 and 4.2.
  const bool two = a.c.d.kv_heads % 2 == 0 && a.rows_max >= kAppendCtas * num_sms();
  return two ? append<T, kI8, 64, 2>(a) : append<T, kI8, 64, 1>(a);
}

}  // namespace

cudaError_t launch_kv8_append(const KvDims& d, const KvState& s, const Kv8Scales& q, int layer, const void* k,
                              const void* v, rpp_dtype dtype, int row_stride, const int32_t* slots, const int32_t* cu, int n,
                              int rows_max, int32_t* err, cudaStream_t stream) {
  const AppendCall a{codes_of(d, s, q, layer), &s, k, v, row_stride, slots, cu, n, rows_max, err, stream};
  if (dtype == RPP_F16) return q.i8 ? append<__half, true>(a) : append<__half, false>(a);
  return q.i8 ? append<__nv_bfloat16, true>(a) : append<__nv_bfloat16, false>(a);
}

cudaError_t launch_kv_read(const KvDims& d, const KvState& s, const Kv8Scales* q, int layer, const int32_t* slots,
                           const int32_t* starts, const int32_t* cu, int n, int rows_max, void* k, void* v,
                           rpp_dtype dtype, int row_stride, int32_t* err, cudaStream_t stream) {
  // Up to 32 rows a warp one wave of warps, with equal shares of the rows.  16281 rows of 8 heads, d = 128: 20.8 us, in two
  // waves 23.4; with a fourth CTA an SM (64 registers, four vectors fewer on their way) 59900 rows take 72 us instead of 66.
  // Above that (116000 rows) up to 8 CTAs an SM that come as others go, not one wave that strides: 300000 rows of 8 heads
  // 302 us, one wave 316; 16 heads, d = 64, 312 and 336; 2 heads, d = 128, 112 and 110.
  const long long warps = static_cast<long long>(kReadCtas) * num_sms() * kMoveWarps;
  const long long passes = (rows_max + warps * kMaxTok - 1) / (warps * kMaxTok);
  const int tok = static_cast<int>((rows_max + warps * passes - 1) / (warps * passes));
  const long long items = (static_cast<long long>(rows_max) + tok - 1) / tok;
  const int grid = blocks_for((items + kMoveWarps - 1) / kMoveWarps, 8 * num_sms());
  const size_t smem = (static_cast<size_t>(n) + 1) * 4;
  const int vpr = d.head_dim / 8;
  int vshift = -1;
  for (int x = 0; x <= 5; ++x)
    if (vpr == 1 << x) vshift = x;
  const int32_t *table = s.table, *lens = s.lens;
  auto go = [&](auto kernel, const Codes& c, auto* ko, auto* vo) {
    return launch_pdl(kernel, dim3(grid), dim3(kMoveThreads), smem, stream, c, table, lens, slots, starts, cu, n, rows_max,
                      tok, vshift, ko, vo, row_stride, err);
  };
  if (!q) {
    Codes c{d, static_cast<uint8_t*>(s.pool), nullptr, 0};
    c.pool += static_cast<size_t>(layer) * d.pages * 2 * d.kv_heads * d.page_size * d.head_dim * 2;
    return go(kv_read_kernel<__half, kPlain16>, c, static_cast<__half*>(k), static_cast<__half*>(v));
  }
  const Codes c = codes_of(d, s, *q, layer);
  if (dtype == RPP_F16)
    return go(q->i8 ? kv_read_kernel<__half, kInt8> : kv_read_kernel<__half, kE4m3>, c, static_cast<__half*>(k),
              static_cast<__half*>(v));
  return go(q->i8 ? kv_read_kernel<__nv_bfloat16, kInt8> : kv_read_kernel<__nv_bfloat16, kE4m3>, c,
            static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v));
}

}  // namespace rpp
