// Writing rows into a quantised key-value cache, and reading rows of any cache back.
//
// Write: x = code * 2^(b - 127) with one byte b for each `block` tokens of a head (code8.cuh).  With a the largest magnitude
// of a block's new rows,
//   b = the smallest byte at which a is no more than half a step past the largest code,
//       or the block's own where it has rows already and that is larger;
//   code = x * 2^(127 - b), rounded half to even; codes the block has are rounded again where b grew.
// Two bytes in and one out per value and no reuse: bound by HBM.  A warp takes one head's K or V of up to 16 rows (or one
// block, if that is longer): it holds the rows in registers, 16 bytes a lane and row, reduces the magnitudes as
// 16-bit integers (their order is the values', and what is not finite is largest), and writes codes and scale.  So
// the rows are read once; only blocks of 32 and more tokens take their rows from L2 a second time.
// All rows of a block that a call brings are one warp's: no atomics, and results do not depend on timing.
//
// Read: a flat copy of rows that turns codes into values on the way, one byte in and two out.
#include "code8.cuh"
#include "kv_common.cuh"

namespace rpp {

namespace {

constexpr int kMoveWarps = kMoveThreads / 32;
constexpr int kMaxTok = 32;     // packed rows that a CTA takes at a time (a lane each of its first warp)

// The packed row t of a call: its sequence, and how far from its end (1: the last token; below 1: nobody's row).
__device__ __forceinline__ int row_owner(const int32_t* __restrict__ cu, int n, int t, long long* back) {
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

// what one warp writes for each head: rows of one 16 (or one longer block) of a page
struct Tile {
  long long page;
  int at;                     // the first row's place in the page
  int rows;
  int t;                      // its packed row
  int lead;                   // rows that its block has already
};

__device__ __forceinline__ uint32_t umax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// the largest magnitude of eight values, as the bits of one
__device__ __forceinline__ uint32_t most8(const uint4& v) {
  const uint32_t m = umax2(umax2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), umax2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}
template <typename T>
__device__ __forceinline__ float of_bits(uint32_t b) {
  const unsigned short s = static_cast<unsigned short>(b);
  return to_f32(*reinterpret_cast<const T*>(&s));
}

// kFine: blocks of fewer than 16 tokens
template <typename T, bool kI8, int D, bool kFine>
__global__ void __launch_bounds__(kMoveThreads)
    kv8_append_kernel(Codes c, const int32_t* __restrict__ table, const int32_t* __restrict__ lens,
                      const int32_t* __restrict__ refs, const T* __restrict__ k, const T* __restrict__ v, int row_stride,
                      const int32_t* __restrict__ slots, const int32_t* __restrict__ cu, int n, int rows_max, int tok,
                      int32_t* err) {
  constexpr int LPR = D / 8;            // lanes of a row
  constexpr int RPS = 32 / LPR;         // rows of a step
  constexpr int S = 16 / RPS;           // steps of 16 rows
  extern __shared__ uint32_t s_seen[];
  __shared__ Gate gate;
  __shared__ Tile s_tile[kMaxTok];
  __shared__ int s_tiles;
  pdl_wait();
  pdl_trigger();
  const int first = static_cast<int>(threadIdx.x) < n ? slots[threadIdx.x] : 0;
  const int T_rows = cu ? cu[n] : n, start = cu ? cu[0] : 0;
  const bool mine = cu && static_cast<int>(threadIdx.x) < n;
  const int c0 = mine ? cu[threadIdx.x] : 0, c1 = mine ? cu[threadIdx.x + 1] : 0;
  if (!pass(slots, n, first, c.d, s_seen, &gate, err, cu, c0, c1)) return;
  if (start < 0 || T_rows > rows_max) {
    if (threadIdx.x == 0) set_device_error(err, RPP_DERR_ROWS);
    return;
  }
  const int ps = c.d.page_size, heads = c.d.kv_heads;
  const int block = 1 << c.shift, unit = kFine || block < 16 ? 16 : block;    // rows of a tile at most
  const int head_scales = ps >> c.shift;
  const long long head_bytes = static_cast<long long>(ps) * D;
  const int warp = warp_id(), lane = lane_id();
  const int lr = lane / LPR, lc = lane % LPR;
  const int chunks = (T_rows + tok - 1) / tok;
  for (int ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
    const int t0 = ch * tok;
    if (warp == 0) {
      bool lead = false;
      Tile x{};
      const int t = t0 + lane;
      if (lane < tok && t < T_rows) {
        long long back;
        const int i = row_owner(cu, n, t, &back);
        const int s = slots[i], len = lens[s];
        if (!len_ok(len, c.d) || back < 1 || back > len) {
          set_device_error(err, RPP_DERR_LENGTH);
        } else {
          const int pos = static_cast<int>(len - back);
          const bool begin = !cu || t == cu[i];
          if (begin || pos % unit == 0) {
            const int p = table[static_cast<long long>(s) * c.d.max_pages + pos / ps];
            if (p < 0 || p >= c.d.pages || refs[p] != 1) {    // not its own page
              set_device_error(err, RPP_DERR_PAGE);
            } else {
              lead = true;
              x.page = p;
              x.at = pos % ps;
              x.rows = static_cast<int>(min(back, static_cast<long long>(unit - pos % unit)));
              x.t = t;
              x.lead = begin ? pos & (block - 1) : 0;
            }
          }
        }
      }
      const uint32_t who = __ballot_sync(0xffffffffu, lead);
      if (lead) s_tile[__popc(who & ((1u << lane) - 1u))] = x;
      if (lane == 0) s_tiles = __popc(who);
    }
    __syncthreads();
    const int jobs = s_tiles * 2 * heads;
    for (int job = warp; job < jobs; job += kMoveWarps) {
      const int ti = job / (2 * heads), kh = job - ti * 2 * heads;    // kh: K's heads, then V's
      const Tile x = s_tile[ti];
      const int o0 = x.at & (unit - 1), o1 = o0 + x.rows;             // the new rows' places in the tile
      const int r0 = x.at - o0;                                       // the tile's place in the page
      const long long head = x.page * 2 * heads + kh;
      uint8_t* codes = c.pool + head * head_bytes + static_cast<long long>(r0) * D;
      uint8_t* scales = c.scales + head * head_scales + (r0 >> c.shift);
      const T* src = (kh < heads ? k : v) + (static_cast<long long>(x.t) - o0) * row_stride +
                     (kh < heads ? kh : kh - heads) * D + lc * 8;
      const int b0 = o0 >> c.shift;                                   // the block that may have rows
      const int had = x.lead ? scales[b0] : 0;
      uint4 w[S];
      auto load = [&](int base) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const int o = base + s * RPS + lr;
          w[s] = make_uint4(0u, 0u, 0u, 0u);
          if (o >= o0 && o < o1) w[s] = *reinterpret_cast<const uint4*>(src + static_cast<long long>(o) * row_stride);
        }
      };
      auto store = [&](int base, const int* b) {
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const int o = base + s * RPS + lr;
          if (o < o0 || o >= o1) continue;
          if (b[s] == 255) w[s] = make_uint4(0u, 0u, 0u, 0u);
          const float inv = b[s] == 255 ? 0.f : inverse_of(b[s]);
          float f[8];
          unpack16<T>(w[s], f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= inv;
          *reinterpret_cast<uint2*>(codes + static_cast<long long>(o) * D + lc * 8) =
              make_uint2(encode4<kI8>(f[0], f[1], f[2], f[3]), encode4<kI8>(f[4], f[5], f[6], f[7]));
        }
      };
      int b[S];                 // scale bytes of the rows in hand
      int lead_b;               // and of the block that may have rows
      if constexpr (kFine) {
        load(0);
        uint32_t m[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
          m[s] = most8(w[s]);
#pragma unroll
          for (int q = LPR / 2; q > 0; q >>= 1) m[s] = max(m[s], __shfl_xor_sync(0xffffffffu, m[s], q));
#pragma unroll
          for (int q = 1; q < RPS; q <<= 1)     // the rows of a step that share a block
            if (q < block) m[s] = max(m[s], __shfl_xor_sync(0xffffffffu, m[s], q * LPR));
        }
#pragma unroll
        for (int q = 1; q < S; q <<= 1) {       // the steps that do
          if (q * RPS >= block) break;
          uint32_t z[S];
#pragma unroll
          for (int s = 0; s < S; ++s) z[s] = max(m[s], m[s ^ q]);
#pragma unroll
          for (int s = 0; s < S; ++s) m[s] = z[s];
        }
        lead_b = 0;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const int o = s * RPS + lr;
          const bool shares = x.lead && (o >> c.shift) == b0;
          b[s] = scale_byte<kI8>(of_bits<T>(m[s]));
          if (shares) {
            b[s] = max(b[s], had);
            lead_b = b[s];
          }
        }
        if (x.lead) lead_b = __reduce_max_sync(0xffffffffu, lead_b);
      } else {
        const int first16 = o0 & ~15, last16 = (o1 - 1) & ~15;
        uint32_t m = 0;
        for (int base = first16; base <= last16; base += 16) {
          load(base);
#pragma unroll
          for (int s = 0; s < S; ++s) m = max(m, most8(w[s]));
        }
        m = __reduce_max_sync(0xffffffffu, m);
        lead_b = max(scale_byte<kI8>(of_bits<T>(m)), had);
#pragma unroll
        for (int s = 0; s < S; ++s) b[s] = lead_b;
      }
      if (x.lead && lead_b > had && lead_b != 255) {    // (a byte of 255 stays for the block's life)
        const float f = pow2_neg(lead_b - had);
        uint4* old = reinterpret_cast<uint4*>(codes + static_cast<long long>(b0 << c.shift) * D);
        const int vecs = x.lead * (D / 16);
#pragma unroll 4
        for (int e = lane; e < vecs; e += 32) {
          uint4 z = old[e];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const float4 y = decode4f<kI8>((&z.x)[h]);
            (&z.x)[h] = encode4<kI8>(y.x * f, y.y * f, y.z * f, y.w * f);
          }
          old[e] = z;
        }
      }
      if constexpr (kFine) {
        store(0, b);
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const int o = s * RPS + lr;
          if (lc == 0 && o >= o0 && o < o1 && o == max(o0, o & ~(block - 1))) scales[o >> c.shift] = static_cast<uint8_t>(b[s]);
        }
      } else {
        const int first16 = o0 & ~15, last16 = (o1 - 1) & ~15;
        for (int base = last16; base >= first16; base -= 16) {    // the last 16 are in hand
          if (base != last16) load(base);
          store(base, b);
        }
        if (lane == 0) scales[b0] = static_cast<uint8_t>(lead_b);
      }
    }
    __syncthreads();   // s_tile is rewritten for the next rows
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

// Rows of K and V of the sequences in `slots` to packed rows.  A lane takes 16 bytes of the pool at a time, four in flight;
// a row of fewer vectors than a warp has lanes shares the warp with the next rows.
template <typename TO, int kCode>
__global__ void __launch_bounds__(kMoveThreads)
    kv_read_kernel(Codes c, const int32_t* __restrict__ table, const int32_t* __restrict__ lens,
                   const int32_t* __restrict__ slots, const int32_t* __restrict__ starts, const int32_t* __restrict__ cu,
                   int n, int rows_max, int tok, TO* __restrict__ k, TO* __restrict__ v, int row_stride, int32_t* err) {
  constexpr int E = kCode == kPlain16 ? 8 : 16;     // values of a vector
  __shared__ int s_flag;
  __shared__ int2 s_row[kMaxTok];                   // page (-1: none) and row in it
  pdl_wait();
  pdl_trigger();
  const int T_rows = cu ? cu[n] : n, start = cu ? cu[0] : 0;
  int bad = 0;
  for (int i = threadIdx.x; i < n; i += kMoveThreads) {
    const int s = slots[i];
    if (s < 0 || s >= c.d.slots) bad |= 2;
    if (cu && cu[i + 1] < cu[i]) bad |= 1;
  }
  if (quit(err, &s_flag)) return;
  const int wrong = __syncthreads_or(bad & 2), back_step = __syncthreads_or(bad & 1);
  if (wrong || back_step || start < 0 || T_rows > rows_max) {
    if (threadIdx.x == 0) set_device_error(err, wrong ? RPP_DERR_SLOT : back_step ? RPP_DERR_LENGTH : RPP_DERR_ROWS);
    return;
  }
  const int ps = c.d.page_size, heads = c.d.kv_heads;
  const int vpr = c.d.head_dim / E;                 // vectors of a head's row
  const int half = heads * vpr, per = 2 * half;
  const int head_scales = ps >> c.shift;
  const uint4* pool = reinterpret_cast<const uint4*>(c.pool);
  const int warp = warp_id(), lane = lane_id();
  const int group = per < 32 ? 32 / per : 1;        // rows that a warp takes at once
  const int lr = per < 32 ? lane / per : 0, lc = per < 32 ? lane - lr * per : lane;
  const int chunks = (T_rows + tok - 1) / tok;
  for (int ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
    const int t0 = ch * tok, have = min(tok, T_rows - t0);
    if (static_cast<int>(threadIdx.x) < have) {
      const int t = t0 + threadIdx.x;
      long long back;
      const int i = row_owner(cu, n, t, &back);
      const int s = slots[i], len = lens[s];
      const long long pos = starts ? static_cast<long long>(starts[i]) + (cu ? t - cu[i] : 0) : len - back;
      int2 at = make_int2(-1, 0);
      if (!len_ok(len, c.d) || back < 1 || pos < 0 || pos >= len || (starts && starts[i] < 0)) {
        set_device_error(err, RPP_DERR_LENGTH);
      } else {
        const int q = static_cast<int>(pos);
        const int p = table[static_cast<long long>(s) * c.d.max_pages + q / ps];
        if (p < 0 || p >= c.d.pages) set_device_error(err, RPP_DERR_PAGE);
        else at = make_int2(p, q % ps);
      }
      s_row[threadIdx.x] = at;
    }
    __syncthreads();
    for (int r0 = warp * group; r0 < have; r0 += kMoveWarps * group) {
      const int r = r0 + lr;
      const int2 at = r < have && lr < group ? s_row[r] : make_int2(-1, 0);
      if (at.x < 0) continue;
      const long long page_head = static_cast<long long>(at.x) * 2 * heads;
      const long long out_row = static_cast<long long>(t0 + r) * row_stride;
      constexpr int U = 4;
      for (int v0 = lc; v0 < per; v0 += U * 32) {
        uint4 x[U];
        int b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int w = v0 + u * 32;
          if (w >= per || (u && per < 32)) continue;
          const int kh = w / vpr;                   // K's heads, then V's
          x[u] = pool[((page_head + kh) * ps + at.y) * vpr + (w - kh * vpr)];
          if constexpr (kCode != kPlain16) b[u] = c.scales[(page_head + kh) * head_scales + (at.y >> c.shift)];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int w = v0 + u * 32;
          if (w >= per || (u && per < 32)) continue;
          uint4* to = reinterpret_cast<uint4*>((w < half ? k + w * E : v + (w - half) * E) + out_row);
          if constexpr (kCode == kPlain16) {
            to[0] = x[u];
          } else {
            const float f = scale_of(b[u]);
            uint4 o[2];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const float4 y = decode4f<kCode == kInt8>((&x[u].x)[h]);
              (&o[h >> 1].x)[2 * (h & 1)] = pack_sat(y.x * f, y.y * f, TO{});
              (&o[h >> 1].x)[2 * (h & 1) + 1] = pack_sat(y.z * f, y.w * f, TO{});
            }
            to[0] = o[0];
            to[1] = o[1];
          }
        }
        if (per < 32) break;
      }
    }
    __syncthreads();   // s_row is rewritten for the next rows
  }
}

// rows a CTA takes at a time: enough CTAs for the grid first, then enough rows for the list check to pay
inline int rows_at_a_time(int rows_max) {
  const int tok = (rows_max + 4 * num_sms() - 1) / (4 * num_sms());
  return tok < 1 ? 1 : tok > kMaxTok ? kMaxTok : tok;
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

template <typename T, bool kI8, int D>
cudaError_t append(const AppendCall& a) {
  const size_t smem = static_cast<size_t>((a.c.d.slots + 31) / 32) * 4;
  const int tok = rows_at_a_time(a.rows_max);
  const int grid = blocks_for((static_cast<long long>(a.rows_max) + tok - 1) / tok, 8 * num_sms());
  return launch_pdl(a.c.shift < 4 ? kv8_append_kernel<T, kI8, D, true> : kv8_append_kernel<T, kI8, D, false>, dim3(grid),
                    dim3(kMoveThreads), smem, a.stream, a.c, static_cast<const int32_t*>(a.s->table),
                    static_cast<const int32_t*>(a.s->lens), static_cast<const int32_t*>(a.s->refs),
                    static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.row_stride, a.slots, a.cu, a.n, a.rows_max,
                    tok, a.err);
}
template <typename T, bool kI8>
cudaError_t append(const AppendCall& a) {
  return a.c.d.head_dim == 64 ? append<T, kI8, 64>(a) : append<T, kI8, 128>(a);
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
  const int tok = rows_at_a_time(rows_max);
  const int grid = blocks_for((static_cast<long long>(rows_max) + tok - 1) / tok, 8 * num_sms());
  const int32_t *table = s.table, *lens = s.lens;
  auto go = [&](auto kernel, const Codes& c, auto* ko, auto* vo) {
    return launch_pdl(kernel, dim3(grid), dim3(kMoveThreads), 0, stream, c, table, lens, slots, starts, cu, n, rows_max, tok,
                      ko, vo, row_stride, err);
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
