// Shared by the attention kernels over the 8-bit paged cache (attn_kv8.cu, attn_kv8_tc.cu): the work
// list and its runs, the partials and their join.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "host_util.h"
#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace batq {

// (the kernels' files each have their own copies of the templates below)
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
  const void* Q;
  int T, ldq, q_heads, kv_heads, group;
  const int* cu_q;
  const int* seq_lens;
  const int* page_table;
  int batch, max_pages, num_pages, page_size, page_shift;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  float scale_log2;
  int max_q_len;
  int runs;            // CTAs of the main kernel
  float* partial;      // [2 * runs][rows][D], then m and l: [2 * runs][rows] each
  int out_bf16;
  void* out;
  int ldo;
  float* lse;
  unsigned* err;
};

// Work units of sequence b (none without queries): kv_heads * row tiles items, each of its key blocks and,
// ahead of them, C::kOver units without keys that stand for what an item costs beside its keys.
struct Items {
  SeqRows s;       // count: the queries to compute
  int queries;     // all of the sequence's, which places them
  int row_tiles, key_blocks, item;
  __device__ int units(int kv_heads) const { return kv_heads * row_tiles * item; }
};
template <class C>
__device__ __forceinline__ Items items_of(const AttnArgs& a, int b) {
  Items it;
  it.s = seq_rows(a.cu_q, a.seq_lens, b, a.T, a.max_pages * a.page_size);
  it.s.len = max(it.s.len, 0);
  it.queries = it.s.count;
  it.s.count = min(it.s.count, a.max_q_len);
  it.row_tiles = (it.s.count * a.group + C::kRows - 1) / C::kRows;
  it.key_blocks = max(1, (it.s.len + C::kUnit - 1) / C::kUnit);  // an empty sequence still writes its zeros
  it.item = it.key_blocks + C::kOver;
  return it;
}

// The W units of the list in R runs of W / R, the first W % R of them one longer.
struct Runs {
  int count, size, longer;
  __device__ int begin(int r) const { return r * size + min(r, longer); }
  // Run of unit u.
  __device__ int of(int u) const {
    const int head = longer * (size + 1);
    return u < head ? u / (size + 1) : longer + (u - head) / size;
  }
};
__device__ __forceinline__ Runs runs_of(int W, int runs) {
  Runs r;
  r.count = min(W, runs);
  r.size = W / max(r.count, 1);
  r.longer = W - r.size * r.count;
  return r;
}

// Units in all, and those before sequence b, by one warp (every lane gets them).
template <class C>
__device__ __forceinline__ int2 count_units(const AttnArgs& a, int b, int lane) {
  int w = 0, before = 0;
  for (int q = lane; q < a.batch; q += 32) {
    const int n = items_of<C>(a, q).units(a.kv_heads);
    w += n;
    before += q < b ? n : 0;
  }
  return make_int2(__reduce_add_sync(0xffffffffu, w), __reduce_add_sync(0xffffffffu, before));
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Sums and outputs count from a reference, the largest of score plus V exponent ev, where ev takes part up to
// +-kFarExp: a reference then is within kFarExp of the scores' own largest, and neither a sum nor the weights that it
// is taken from leave fp32's range (a weight is 0 at 2^-141 of the largest: -141 + 2 * 56 = -29, below a sum's 24
// bits).  Sums counted from exponents up to 127 lost the tokens of pages with small values beside ones with large
// values, and all of themselves at a change of reference.
constexpr float kFarExp = 56.0f;
__device__ __forceinline__ float near_exponent(float ev) { return fminf(fmaxf(ev, -kFarExp), kFarExp); }

// 2^e as a product of two: v * 2^e may be in fp32's range where 2^e is not.
struct Pow2 {
  float a, b;
};
__device__ __forceinline__ Pow2 pow2_of(float e) {
  e = fmaxf(e, -250.0f);  // (also -inf)
  const float h = floorf(0.5f * e);
  return Pow2{ex2(h), ex2(e - h)};
}
__device__ __forceinline__ float times(float v, Pow2 p) { return v * p.a * p.b; }

// Bit 7 of every byte that is an E4M3 NaN (all of its low seven bits set).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Joins the partials of the items cut by run borders.  kJW warps per row take its partials in turn
// (warp w every kJW-th, in key order), then their sums are added in order.
constexpr int kJoinWarps = 8;
template <class C, int kJW>
__global__ void __launch_bounds__(32 * kJoinWarps) k_attn_kv8_join(const AttnArgs a, const int most_rows) {
  constexpr int kD = C::kD, kRows = C::kRows, kPer = kD / 32, kRowsPerCta = kJoinWarps / kJW;
  __shared__ float s_acc[kJoinWarps][kD];
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, slot = threadIdx.x >> 5, warp = slot % kJW, first = slot - warp;
  const int b = blockIdx.y, x = blockIdx.x * kRowsPerCta + slot / kJW;
  const int h = x / most_rows, rr = x - h * most_rows;  // kv head, row of the (sequence, kv head)
  const Items it = items_of<C>(a, b);
  if (h >= a.kv_heads || rr >= it.s.count * a.group) return;  // (all warps of a row together)
  const int rt = rr / kRows, r = rr - rt * kRows;
  const int2 W = count_units<C>(a, b, lane);
  const Runs runs = runs_of(W.x, a.runs);
  const int u0 = W.y + (h * it.row_tiles + rt) * it.item;
  const int r0 = runs.of(u0 + C::kOver), r1 = runs.of(u0 + it.item - 1);
  if (r0 == r1) return;  // written by its CTA
  const int slot0 = 2 * r0 + (runs.begin(r0) >= u0 ? 0 : 1);
  const float* ml = a.partial + (size_t)2 * a.runs * kRows * kD;
  const float* ll = ml + (size_t)2 * a.runs * kRows;
  float mx = -INFINITY, sum = 0.0f, acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
  constexpr int kFlight = kJW == 1 ? 4 : 8;  // partials in flight per warp
  for (int c0 = r0 + warp; c0 <= r1; c0 += kFlight * kJW) {
    float pm[kFlight], pl[kFlight], v[kFlight][kPer];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int c = c0 + k * kJW;
      pm[k] = -INFINITY;
      pl[k] = 0.0f;
      if (c <= r1) {
        const size_t at = (size_t)(c == r0 ? slot0 : 2 * c) * kRows + r;
        pm[k] = ml[at];
        pl[k] = ll[at];
#pragma unroll
        for (int i = 0; i < kPer; i += 2) {
          const float2 x = *reinterpret_cast<const float2*>(a.partial + at * kD + lane * kPer + i);
          v[k][i] = x.x;
          v[k][i + 1] = x.y;
        }
      }
    }
    float m_new = mx;
#pragma unroll
    for (int k = 0; k < kFlight; ++k) m_new = fmaxf(m_new, pm[k]);
    // Without any maximum there is nothing to weigh (sums of zero, or of NaN).
    const Pow2 alpha = pow2_of(m_new == -INFINITY ? 0.0f : mx - m_new);
    sum = times(sum, alpha);
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = times(acc[i], alpha);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (c0 + k * kJW > r1) break;
      const Pow2 w = pow2_of(m_new == -INFINITY ? 0.0f : pm[k] - m_new);
      sum = fmaf(w.a * pl[k], w.b, sum);
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] = fmaf(w.a * v[k][i], w.b, acc[i]);
    }
    mx = m_new;
  }
  const size_t row = (size_t)(it.s.begin + rr / a.group);
  const int head = h * a.group + rr % a.group;
  const size_t o = row * (size_t)a.ldo + (size_t)head * kD;
  if constexpr (kJW > 1) {
    if (lane == 0) {
      s_m[slot] = mx;
      s_l[slot] = sum;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) s_acc[slot][lane * kPer + i] = acc[i];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + first / kJW), "n"(32 * kJW) : "memory");
    if (warp != 0) return;
    mx = s_m[first];
#pragma unroll
    for (int w = 1; w < kJW; ++w) mx = fmaxf(mx, s_m[first + w]);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < kJW; ++w) {
      const Pow2 weight = pow2_of(mx == -INFINITY ? 0.0f : s_m[first + w] - mx);
      sum = fmaf(weight.a * s_l[first + w], weight.b, sum);
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] = fmaf(weight.a * s_acc[first + w][lane * kPer + i], weight.b, acc[i]);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : C::kOutUnit / sum;  // a row that sees nothing: zeros
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {
    if (a.out_bf16)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + o + lane * kPer + i) =
          pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
    else
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + o + lane * kPer + i) =
          make_float2(acc[i] * inv, acc[i + 1] * inv);
  }
  if (a.lse && lane == 0) a.lse[row * a.q_heads + head] = sum == 0.0f ? -INFINITY : kLn2 * (mx + log2f(sum));
}

// Arguments of a launch, and the join after it: `unit` keys per work unit, `rows` the kernel's row tile.
inline AttnArgs attn_args(const AttnKv8Launch& L, int runs) {
  AttnArgs a = {};
  a.Q = L.Q;
  a.T = L.T;
  a.ldq = L.ldq;
  a.q_heads = L.q_heads;
  a.kv_heads = L.kv_heads;
  a.group = L.q_heads / L.kv_heads;
  a.cu_q = L.cu_q;
  a.seq_lens = L.seq_lens;
  a.page_table = L.page_table;
  a.batch = L.batch;
  a.max_pages = L.max_pages;
  a.num_pages = L.num_pages;
  a.page_size = L.page_size;
  a.page_shift = L.page_size == 16 ? 4 : L.page_size == 32 ? 5 : L.page_size == 64 ? 6 : 7;
  a.k_scales = L.k_scales;
  a.v_scales = L.v_scales;
  a.scale_log2 = L.softmax_scale * kLog2e;
  a.max_q_len = L.max_q_len;
  a.partial = L.workspace;
  a.out_bf16 = L.out_bf16 ? 1 : 0;
  a.out = L.out;
  a.ldo = L.ldo;
  a.lse = L.lse;
  a.err = L.err;
  a.runs = runs;
  return a;
}

constexpr int kMaxRuns = 592;  // 148 SMs x 4 CTAs

template <class C>
cudaError_t launch_join(const AttnKv8Launch& L, const AttnArgs& a, cudaStream_t stream) {
  // No sequence can be longer than its page table: when that is one unit, no item is ever cut.
  if ((long long)L.max_pages * L.page_size <= C::kUnit) return cudaSuccess;
  const long long rows_most = (long long)L.max_q_len * a.group, rows_all = rows_most * L.kv_heads;
  // With at least a quarter as many items as runs an item has about four partials at most: a warp per row.
  const bool few = (long long)L.batch * L.kv_heads * 4 >= a.runs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(few ? (rows_all + kJoinWarps - 1) / kJoinWarps : rows_all), (unsigned)L.batch);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&cfg, k_attn_kv8_join<C, 1>, a, (int)rows_most)
             : cudaLaunchKernelEx(&cfg, k_attn_kv8_join<C, kJoinWarps>, a, (int)rows_most);
}

}  // namespace

// Head dim 128 and long sequences, on the 5th-generation tensor cores (attn_kv8_tc.cu).
cudaError_t launch_attn_kv8_tc(const AttnKv8Launch& L, cudaStream_t stream);

}  // namespace batq
