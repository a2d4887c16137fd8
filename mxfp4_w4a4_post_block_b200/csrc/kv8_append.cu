// k_kv8_append: new K and V rows into the pages of an 8-bit cache with one scale per (page, kv head).
//
// A block of the cache is one head's rows of one page.  Its scale is 2^e with the smallest e that
// covers every finite value written to the block so far (amax <= 448 * 2^e, so nothing saturates);
// codes are E4M3_RNE(x * 2^-e).  A power of two costs E4M3 no precision (its step is relative) and
// makes the scale's growth exact: when a later token needs a larger e, the block's older codes are
// multiplied by 2^(e_old - e) and rounded again, which is exact down to the E4M3 subnormals.  The
// first token of a page sets the scale afresh, whatever the page held before.  NaN and infinities
// are stored as the E4M3 NaN and take no part in the amax.
//
// One CTA owns one block that receives tokens (blockIdx.x: the touched pages of the batch in order;
// y: kv head; z: K or V), so no block has two writers and the result does not depend on order.  Up to
// eight 8-element chunks per thread (64 rows of 128) are loaded together and stay in registers from the
// maximum to the codes; larger blocks are read twice, eight chunks at a time, the second time from L2.
// (One chunk at a time, each with its own trip to memory: 23.7 us for 8000 rows of 8 x 128 instead of
// 17.1.)  The maximum is taken of the bits as integers, two bf16 at a time, and values are checked for NaN and
// infinities only where that maximum shows some (17.2 -> 15.1 us; memory 11.3).  One token of 64 sequences: 4.3 us,
// the launch and three dependent reads.
#include <cstdint>
#include <type_traits>

#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace batq {
namespace {

constexpr int kThreads = 128;
constexpr int kPiece = 8;  // chunks in flight per thread

// Smallest e >= -127 with |a| <= 448 * 2^e (448 = 1.75 * 2^8), a finite and >= 0.
__device__ __forceinline__ int block_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(e, -127);
}

__device__ __forceinline__ float finite_or_nan(float v) {
  return fabsf(v) <= 3.402823466e38f ? v : __uint_as_float(0x7FC00000u);
}

// Eight consecutive elements of a row, as loaded.
template <bool kBF16>
struct Raw8 {
  uint4 q[kBF16 ? 1 : 2];
};
template <bool kBF16>
__device__ __forceinline__ Raw8<kBF16> load8(const uint8_t* p) {
  Raw8<kBF16> r;
#pragma unroll
  for (int i = 0; i < (kBF16 ? 1 : 2); ++i) r.q[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
template <bool kBF16>
__device__ __forceinline__ void values8(const Raw8<kBF16>& r, float (&v)[8]) {
  if constexpr (kBF16) {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[4 * i] = __uint_as_float(r.q[i].x);
      v[4 * i + 1] = __uint_as_float(r.q[i].y);
      v[4 * i + 2] = __uint_as_float(r.q[i].z);
      v[4 * i + 3] = __uint_as_float(r.q[i].w);
    }
  }
}

// Largest magnitude of eight elements as loaded and `top`, as fp32 bits (without the sign they are ordered as
// integers; two bf16 at a time).
template <bool kBF16>
__device__ __forceinline__ uint32_t max8(const Raw8<kBF16>& r, uint32_t top) {
  if constexpr (kBF16) {
    const uint32_t m = __vmaxu2(__vmaxu2(r.q[0].x & 0x7FFF7FFFu, r.q[0].y & 0x7FFF7FFFu),
                                __vmaxu2(r.q[0].z & 0x7FFF7FFFu, r.q[0].w & 0x7FFF7FFFu));
    return max(top, max(m << 16, m & 0xFFFF0000u));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      top = max(max(top, max(r.q[i].x & 0x7FFFFFFFu, r.q[i].y & 0x7FFFFFFFu)),
                max(r.q[i].z & 0x7FFFFFFFu, r.q[i].w & 0x7FFFFFFFu));
    return top;
  }
}

// The item-th touched page, by one warp: sequence b with new tokens at positions len - count .. len - 1, or -1.
// `total`: all touched pages, where they are counted.
struct Item {
  int seq, page, total;
};
__device__ __forceinline__ Item find_item(const Kv8AppendLaunch& a, const int item, const bool count_all) {
  const int lane = threadIdx.x & 31, max_len = a.max_pages * a.page_size;
  int before = 0, seq = -1, page = 0;
  for (int b0 = 0; b0 < a.batch && (seq < 0 || count_all); b0 += 32) {
    const int b = b0 + lane;
    int first = 0, n = 0;
    if (b < a.batch) {
      const SeqRows s = seq_rows(a.cu_new, a.seq_lens, b, a.T, max_len);
      if (s.count > 0 && a.seq_lens[b] >= s.count) {  // tokens past the page table are dropped
        first = (a.seq_lens[b] - s.count) / a.page_size;
        n = max(0, (s.len - 1) / a.page_size - first + 1);
      }
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const int at = item - before - (incl - n);
    const unsigned hit = __ballot_sync(0xffffffffu, at >= 0 && at < n);
    if (hit) {
      const int src = __ffs(hit) - 1;
      seq = b0 + src;
      page = __shfl_sync(0xffffffffu, first + at, src);
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return Item{seq, page, count_all ? before : 0};
}

// Writes the new rows of page `page` of sequence b, K's or V's of one head, by the CTA.
template <bool kBF16>
__device__ __forceinline__ void write_block(const Kv8AppendLaunch& a, const int b, const int page, uint32_t* s_top) {
  const int tid = threadIdx.x, lane = tid & 31, max_len = a.max_pages * a.page_size;
  const int pid = a.page_table[(size_t)b * a.max_pages + page];  // (checked once the rows are on their way)
  const SeqRows s = seq_rows(a.cu_new, a.seq_lens, b, a.T, max_len);
  const int pos0 = a.seq_lens[b] - s.count;                      // position of the sequence's first new token
  const int begin = max(pos0, page * a.page_size);               // this page's new positions
  const int end = min(s.len, (page + 1) * a.page_size);
  const int off0 = begin - page * a.page_size;                   // rows that were there before
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int D = a.head_dim, per_row = D >> 3, chunks = (end - begin) * per_row;
  constexpr size_t esz = kBF16 ? 2 : 4;
  const size_t ld = (size_t)(is_v ? a.ldv : a.ldk) * esz;
  const uint8_t* x = static_cast<const uint8_t*>(is_v ? a.V : a.K) + (size_t)(s.begin + begin - pos0) * ld +
                     (size_t)h * D * esz;
  // Chunk c: row c / per_row of the new ones, elements 8 (c % per_row) ..; per_row is a power of two.
  const int row_shift = 31 - __clz(per_row);
  auto load_piece = [&](int c0, Raw8<kBF16> (&raw)[kPiece]) {
#pragma unroll
    for (int j = 0; j < kPiece; ++j) {
      const int c = c0 + j * kThreads;
      if (c < chunks) raw[j] = load8<kBF16>(x + (size_t)(c >> row_shift) * ld + (size_t)(c & (per_row - 1)) * 8 * esz);
    }
  };
  Raw8<kBF16> raw[kPiece];
  load_piece(tid, raw);
  if (pid < 0 || pid >= a.num_pages) return;
  const size_t block = (size_t)pid * a.kv_heads + h;
  uint8_t* codes = (is_v ? a.v_codes : a.k_codes) + block * ((size_t)a.page_size * D);
  uint8_t* scale = (is_v ? a.v_scales : a.k_scales) + block;
  const int e_old = off0 > 0 ? (int)*scale - 127 : -127;
  auto block_max = [&](uint32_t v) {
    v = __reduce_max_sync(0xffffffffu, v);
    if (lane == 0) s_top[tid >> 5] = v;
    __syncthreads();  // the first time also: every thread has the old scale before it is replaced
    v = s_top[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) v = max(v, s_top[i]);
    return v;
  };
  const bool kept = chunks <= kPiece * kThreads;  // the rows stay in registers
  uint32_t top = 0;
  for (int c0 = tid; c0 < chunks; c0 += kPiece * kThreads) {
    if (c0 != tid) load_piece(c0, raw);
#pragma unroll
    for (int j = 0; j < kPiece; ++j)
      if (c0 + j * kThreads < chunks) top = max8<kBF16>(raw[j], top);
  }
  top = block_max(top);
  const bool finite = top < 0x7F800000u;
  if (!finite) {  // the largest of the finite values
    top = 0;
    for (int c0 = tid; c0 < chunks; c0 += kPiece * kThreads) {
      if (!kept) load_piece(c0, raw);
#pragma unroll
      for (int j = 0; j < kPiece; ++j)
        if (c0 + j * kThreads < chunks) {
          float v[8];
          values8<kBF16>(raw[j], v);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t m = __float_as_uint(v[i]) & 0x7FFFFFFFu;
            top = m < 0x7F800000u ? max(top, m) : top;
          }
        }
    }
    __syncthreads();  // s_top has been read
    top = block_max(top);
  }
  const float amax = __uint_as_float(top);
  const int e = max(e_old, block_exponent(amax));
  if (tid == 0) *scale = (uint8_t)(e + 127);

  if (e > e_old && off0 > 0) {
    const float f = e8m0_value((uint32_t)max(127 + e_old - e, 0));
    uint4* old = reinterpret_cast<uint4*>(codes);
    for (int c = tid; c < off0 * D / 16; c += kThreads) {
      const uint4 q = old[c];
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 lo = e4m3x2_values(w[i] & 0xFFFFu), hi = e4m3x2_values(w[i] >> 16);
        r[i] = e4m3x4(lo.x * f, lo.y * f, hi.x * f, hi.y * f);
      }
      old[c] = make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
  const float inv = e8m0_value((uint32_t)max(127 - e, 0));  // 2^-e
  uint8_t* dst = codes + (size_t)off0 * D;
  auto encode = [&](auto checked) {
    for (int c0 = tid; c0 < chunks; c0 += kPiece * kThreads) {
      if (!kept) load_piece(c0, raw);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        const int c = c0 + j * kThreads;
        if (c < chunks) {
          float v[8];
          values8<kBF16>(raw[j], v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = (decltype(checked)::value ? finite_or_nan(v[i]) : v[i]) * inv;
          reinterpret_cast<uint2*>(dst)[c] = make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
        }
      }
    }
  };
  if (finite)
    encode(std::false_type{});
  else
    encode(std::true_type{});
}

template <bool kBF16>
__global__ void __launch_bounds__(kThreads, kBF16 ? 9 : 5) k_kv8_append(const Kv8AppendLaunch a) {
  __shared__ int s_seq, s_page, s_total;
  __shared__ uint32_t s_top[kThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const bool last = blockIdx.x + 1 == gridDim.x;
  auto find = [&](const int item) {
    if (threadIdx.x < 32) {
      const Item x = find_item(a, item, last);
      if (threadIdx.x == 0) {
        s_seq = x.seq;
        s_page = x.page;
        s_total = x.total;
      }
    }
    __syncthreads();
  };
  find(blockIdx.x);
  if (last) {
    // Sequences whose ranges of rows overlap touch more pages than the other CTAs take: this one takes the rest.  (In a
    // branch of its own; as a loop around one copy of the code it took 8000 rows of 8 x 128 from 14.9 to 16.0 us.)
    for (int item = blockIdx.x; item < s_total; ++item) {
      if (s_seq >= 0) write_block<kBF16>(a, s_seq, s_page, s_top);
      __syncthreads();  // what the item shared has been read
      find(item + 1);
    }
    return;
  }
  if (s_seq >= 0) write_block<kBF16>(a, s_seq, s_page, s_top);
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendLaunch& L, cudaStream_t stream) {
  // A sequence with n >= 1 new tokens touches at most min(n, n / page + 2) pages; without ranges that overlap the last
  // CTA has nothing to do.
  const long long items = (long long)L.T / L.page_size + 2LL * L.batch;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items < L.T ? items : L.T) + 1u, (unsigned)L.kv_heads, 2);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return L.bf16 ? cudaLaunchKernelEx(&cfg, k_kv8_append<true>, L) : cudaLaunchKernelEx(&cfg, k_kv8_append<false>, L);
}

}  // namespace batq
