// What the single-token attentions over a paged cache share (attention_decode.cu: 16-bit values,
// attention_decode8.cuh: 8-bit codes): how the work of a call is cut over the warps of the grid, and the kernels that join
// what was cut.  The work is one line of key blocks (sequence, kv head and 16 of its query heads, block), cut into equal
// shares, one a warp; a (sequence, kv head) that several warps had leaves maximum, sum and unnormalised output of each
// in the workspace, and a second kernel joins them in a fixed order.
#pragma once
#include <type_traits>

#include "kernels.h"

namespace rpp {

namespace {

constexpr int kMinBlocks = 2;           // blocks a warp takes at least, while there are that many
constexpr int kRows = 16;               // query heads of a unit
constexpr int kJoinThreads = 128;        // join by cuts
constexpr int kHeadThreads = 256;        // join by heads

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

// The first words of a main kernel: blocks of KB keys before each sequence in s_pre [n + 1] (and in p.prefix, for
// the join), zeros for empty sequences.  Returns the blocks of one kv head part, -1 if the error word was set.
// Holds __syncthreads: called by all threads.
template <typename T, int D, int KB, int W>
__device__ __forceinline__ long long line_plan(const DecodeParams& p, long long* s_pre) {
  __shared__ int s_flag;
  __shared__ long long s_warp[W];
  const int warp = warp_id(), lane = lane_id();
  // one reading of the error word for the whole CTA, on its way together with the first lengths
  if (threadIdx.x == 0) s_flag = device_error_set(p.err) ? 1 : 0;
  int slot0;
  const int len0 = static_cast<int>(threadIdx.x) < p.n ? seq_len(p, threadIdx.x, &slot0) : 0;
  __syncthreads();
  if (s_flag) return -1;

  // ---- blocks before each sequence
  long long carry = 0;
  for (int base = 0; base < p.n; base += W * 32) {
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
    for (int w = 0; w < W; ++w) {
      if (w < warp) before += s_warp[w];
      carry += s_warp[w];
    }
    if (i < p.n) s_pre[i] = before + x - v;
    __syncthreads();
  }
  if (threadIdx.x == 0) s_pre[p.n] = carry;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= p.n; i += W * 32) p.prefix[i] = s_pre[i];
  // empty sequences: zeros
  for (int i = warp * gridDim.x + blockIdx.x; i < p.n; i += W * gridDim.x) {
    if (s_pre[i + 1] != s_pre[i]) continue;
    uint4* row = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + static_cast<long long>(i) * p.nh * D);
    for (int e = lane; e < p.nh * (D / 8); e += 32) row[e] = make_uint4(0u, 0u, 0u, 0u);
  }
  return carry;
}

// A place in the line of blocks.
struct LineCursor {
  int i, unit, blk, nb, len;
  const int32_t* row;            // page numbers of the sequence
  __device__ __forceinline__ void enter(const DecodeParams& p, const long long* s_pre) {   // the lengths of sequence i
    int slot;
    len = seq_len(p, i, &slot);
    nb = static_cast<int>(s_pre[i + 1] - s_pre[i]);
    row = p.table + static_cast<long long>(slot) * p.d.max_pages;
  }
  // block f of the line
  __device__ __forceinline__ void start(const DecodeParams& p, const long long* s_pre, int per_seq, long long f) {
    int lo = 0, hi = p.n - 1;    // the last sequence that starts at or before f (empty ones passed over)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pre[mid] * per_seq <= f) lo = mid;
      else hi = mid - 1;
    }
    i = lo;
    enter(p, s_pre);
    const long long rem = f - s_pre[i] * per_seq;
    unit = static_cast<int>(rem / nb);
    blk = static_cast<int>(rem - static_cast<long long>(unit) * nb);
  }
  // the next block (only while there is one)
  __device__ __forceinline__ void advance(const DecodeParams& p, const long long* s_pre, int per_seq) {
    if (++blk < nb) return;
    blk = 0;
    if (++unit < per_seq) return;
    unit = 0;
    do ++i;
    while (i < p.n - 1 && s_pre[i + 1] == s_pre[i]);
    enter(p, s_pre);
  }
};

// a piece's output by its factor; one that is not finite stays (the factor may have underflowed to 0)
__device__ __forceinline__ float weighted(float a, float x) { return isfinite(x) ? a * x : x; }

// One CTA for each share of the line: if its start is the first cut of a unit, the CTA joins that
// unit's pieces.  A thread has four output elements of one head and, where there are fewer of
// those than threads, one of several groups of pieces.
// kMost > 0: units of about kMost pieces and more (by their sequence's blocks) are left to join_long_units.
template <typename T, int D, int kMost>
__device__ __forceinline__ void join_cut(const DecodeParams& p, int main_warps) {
  __shared__ int s_flag;
  __shared__ float s_m[kRows];
  __shared__ float4 s_o[kJoinThreads];
  __shared__ float s_lg[kJoinThreads];
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
  if (kMost > 0 && nb * warps >= kMost * total) return;
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

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads, 12)
    attention_decode_join_cuts_kernel(const DecodeParams p, int main_warps) {
  pdl_wait();
  pdl_trigger();
  join_cut<T, D, 0>(p, main_warps);
}

inline size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// The workspace of a call whose main kernel has `warps` warps.
inline size_t line_ws_bytes(int n, int nh, int nkv, int d, long long warps) {
  const size_t pieces = 2 * static_cast<size_t>(warps);
  const int group = nh / nkv, kept = group < kRows ? group : kRows;
  return up256((static_cast<size_t>(n) + 1) * sizeof(long long)) + up256(pieces / 2 * sizeof(int4)) +
         up256(pieces * kRows * sizeof(float2)) + up256(pieces * kept * d * sizeof(float));
}
inline void line_ws_bind(DecodeParams* p, void* ws, long long warps) {
  const size_t pieces = 2 * static_cast<size_t>(warps);
  uint8_t* at = static_cast<uint8_t*>(ws);
  p->prefix = reinterpret_cast<long long*>(at);
  at += up256((static_cast<size_t>(p->n) + 1) * sizeof(long long));
  p->cuts = reinterpret_cast<int4*>(at);
  at += up256(pieces / 2 * sizeof(int4));
  p->ml = reinterpret_cast<float2*>(at);
  at += up256(pieces * kRows * sizeof(float2));
  p->acc = reinterpret_cast<float*>(at);
}

// The join after a main kernel of `warps` warps: by query head while they are few (few units of many pieces), else
// one CTA for each place where the line was cut (many units of few pieces).
template <typename T, int D>
cudaError_t launch_join(const DecodeParams& p, int warps, cudaStream_t stream) {
  if (static_cast<long long>(p.n) * p.nh <= 4 * num_sms())
    return launch_pdl(attention_decode_join_heads_kernel<T, D>, dim3(p.n, p.nh), dim3(kHeadThreads), 0, stream, p, warps);
  return launch_pdl(attention_decode_join_cuts_kernel<T, D>, dim3(warps), dim3(kJoinThreads), 0, stream, p, warps);
}

}  // namespace

}  // namespace rpp
