// k_attn_kv8: attention of few queries per sequence over the 8-bit paged cache (kv8.cuh).
//
// For query i of a sequence with n queries and L tokens in the cache (the queries' own among them),
// head h of kv head j = h / G:
//   s_t = scale * 2^ek(t) * <q, K_t>,  t <= L - n + i;   p = softmax(s);   o = sum_t p_t 2^ev(t) V_t
// in one pass over the cache with a running maximum and sum (fp32) per row.
//
// The G heads of a kv head times the queries are the rows of m16n8k16 matrix instructions: rows and
// not keys fill the 16-row side, since K's and V's bytes are what has to move (a decode step does
// about 2 G operations per byte; the tensor pipe idles).  E4M3 widens exactly to f16, so K and V
// enter as f16 codes and the page scales stay outside: 2^ek multiplies the fp32 scores, 2^ev the
// probabilities (below).  Q is rounded to f16 after an exact power-of-two normalisation of its row
// (bf16 queries keep all their bits down to 2^-28 of the row's largest; fp32 queries keep 11);
// probabilities are rounded to f16 (2^-11 relative), less than the bf16 output's own step.
//
// Layout in registers.  The reduction dimensions may be ordered freely, as long as both operands
// agree, so a lane reads 16 consecutive bytes of a K row (one LDS.128 feeds four K steps) and, of V,
// four bytes (head dims) of each of four keys, transposed by byte permutes into the f16 pairs
// (two keys of one head dim) that the instruction wants; the output then has eight consecutive head
// dims per lane.  Tiles of 32 keys come by TMA with the 128-byte (head dim 64: 64-byte) swizzle,
// which makes both reads conflict-free.
//
// Work split.  The keys of all (sequence, kv head, row tile) items are cut into blocks of kUnit keys;
// the list of all blocks is dealt out in equal contiguous runs, one per CTA, computed by each CTA
// from seq_lens.  A CTA whose run covers an item writes its output; items cut by run borders leave
// (m, l, o) partials in the workspace (at most two per CTA: its first and its last item), joined in
// key order by k_attn_kv8_join.  Within a CTA, kKW key groups take every kKW-th tile, each with a
// ring of its own, and kRW warps of a group share its tiles for further rows.
#include <cstdint>

#include "host_util.h"
#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace batq {
namespace {

constexpr int kTile = 32;  // keys per tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// kD: head dim; kMT: 16-row tiles per warp; kRW: row warps; kKW: key groups.
// kCtas: CTAs per SM that registers and shared memory are laid out for.
template <int kD_, int kMT_, int kRW_, int kKW_, int kStages_, int kCtas_>
struct AttnCfg {
  static constexpr int kD = kD_, kMT = kMT_, kRW = kRW_, kKW = kKW_, kStages = kStages_,
                       kCtas = kCtas_;
  static constexpr int kRowsPerWarp = 16 * kMT;
  static constexpr int kRows = kRowsPerWarp * kRW;
  static constexpr int kThreads = 32 * kRW * kKW;
  static constexpr int kUnit = kTile * kKW;                 // keys per work unit
  static constexpr int kBoxD = kD < 128 ? kD : 128;         // bytes per row of one swizzled box
  static constexpr int kHalves = kD / kBoxD;                // boxes along the head dim
  static constexpr int kTileBytes = kTile * kD;
  static constexpr int kStageBytes = 2 * kTileBytes;        // K, V
  static constexpr int kRingBytes = kKW * kStages * kStageBytes;
  static constexpr int kPitch = kD + 4;                     // floats per row of the merge buffer
  static constexpr int kMergeBytes = kKW * kRows * kPitch * 4;
  static constexpr int kDataBytes = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;  // the merge reuses the ring
  static constexpr int kQBytes = kRows * kD * 2;
  static constexpr int kSmallBytes = kRows * 4 + 2 * kKW * kRows * 4 + 2 * kKW * kStages * 8 + kKW * kStages * 32 + 64;
  static constexpr int kSmemBytes = kDataBytes + kQBytes + kSmallBytes + 1024;
};

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
  int min_units;       // shortest run worth a CTA of its own
  float* partial;      // [2 * runs][rows][D], then m and l: [2 * runs][rows] each
  int out_bf16;
  void* out;
  int ldo;
  float* lse;
  unsigned* err;
};

// Work units of sequence b: kv_heads * row tiles * key blocks (none without queries).
struct Items {
  SeqRows s;       // count: the queries to compute
  int queries;     // all of the sequence's, which places them
  int row_tiles, key_blocks;
  __device__ long long units(int kv_heads) const { return (long long)kv_heads * row_tiles * key_blocks; }
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
  return it;
}

// Runs: with W units in all and R runs in use, run r is units [W r / R, W (r + 1) / R).
__device__ __forceinline__ int runs_used(long long W, int runs, int min_units) {
  const long long most = (W + min_units - 1) / min_units;
  return (int)(most < runs ? (most > 0 ? most : 1) : runs);
}

// Sum of all units, by one warp (every lane gets it).
template <class C>
__device__ __forceinline__ long long total_units(const AttnArgs& a, int lane) {
  long long w = 0;
  for (int b = lane; b < a.batch; b += 32) w += items_of<C>(a, b).units(a.kv_heads);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
  return w;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two f16 pairs from four E4M3 bytes (exact): bytes 0, 1 -> lo, bytes 2, 3 -> hi.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// Maximum of three; NaN is passed over.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// V's page scales ride on the scores: with x_t the score in log2 units and 2^ev(t) the scale of token
// t's V block, the weights in the matrix instruction are p_t = 2^(x_t + ev(t) - m + kBias), m the
// running maximum of x + ev, and the sum takes p_t 2^-(ev(t) + kBias) = 2^(x_t - m).  So f16 keeps 11
// bits of every weight that matters beside the row's largest product of probability and scale (the
// bias puts that one at 2^15, and f16's smallest step 2^39 below it) however far apart the blocks'
// scales are, and the accumulators need no unit of their own.  Scales below 2^kMinExp (an all-zero
// block has 2^-127) ride as 2^kMinExp, which keeps the sum inside fp32, and the rest multiplies the
// f16 weights.
constexpr int kBias = 15;
constexpr int kMinExp = -100;
constexpr float kUnbias = 1.0f / 32768.0f;
__device__ __forceinline__ float v_exponent(int byte) {
  return byte == 255 ? __uint_as_float(0x7FC00000u) : (float)max(byte - 127, kMinExp);
}

// Bit 7 of every byte that is an E4M3 NaN (all of its low seven bits set).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

__device__ __forceinline__ uint32_t lds32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
    k_attn_kv8(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const AttnArgs a,
               const int q_bf16) {
  constexpr int kD = C::kD, kMT = C::kMT, kKW = C::kKW, kRW = C::kRW, kStages = C::kStages, kRows = C::kRows;
  extern __shared__ uint8_t smem_raw[];
  // (an offset, so that the compiler still knows these for shared addresses)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_q = smem + C::kDataBytes;                                       // Q fragments (f16)
  float* s_rf = reinterpret_cast<float*>(s_q + C::kQBytes);                  // [kRows] scale of each row's scores
  float* s_m = s_rf + kRows;                                                 // [kKW][kRows]
  float* s_l = s_m + kKW * kRows;                                            // [kKW][kRows]
  uint64_t* s_full = reinterpret_cast<uint64_t*>(s_l + kKW * kRows);         // [kKW][kStages]
  uint64_t* s_empty = s_full + kKW * kStages;                                // [kKW][kStages]
  float4* s_meta = reinterpret_cast<float4*>(s_empty + kKW * kStages);       // [kKW][kStages][2], see fetch

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kw = warp / kRW, rw = warp % kRW;
  const int g = lane >> 2, t = lane & 3;
  if (tid == 0) {
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
    for (int i = 0; i < kKW * kStages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kRW);
    }
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();

  const long long W = total_units<C>(a, lane);
  const int runs = runs_used(W, a.runs, a.min_units);
  if ((int)blockIdx.x >= runs || W == 0) return;
  long long u = W * blockIdx.x / runs;
  const long long u_end = W * (blockIdx.x + 1) / runs;
  const long long u_begin = u;

  // The sequence of unit u: each warp scans the batch.
  int b = 0;
  long long base = 0;  // units before sequence b
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const long long n = b0 + lane < a.batch ? items_of<C>(a, b0 + lane).units(a.kv_heads) : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const bool here = n > 0 && base + incl > u && base + incl - n <= u;
    const unsigned hit = __ballot_sync(0xffffffffu, here);
    if (hit) {
      const int src = __ffs(hit) - 1;
      b = b0 + src;
      base += __shfl_sync(0xffffffffu, incl - n, src);
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }

  uint8_t* ring = smem + kw * (kStages * C::kStageBytes);
  uint64_t* full = s_full + kw * kStages;
  uint64_t* empty = s_empty + kw * kStages;
  float4* meta = s_meta + kw * kStages * 2;
  int p_slot = 0, c_slot = 0;         // producer's and consumer's ring slots
  uint32_t p_phase = 0, c_phase = 0;

  while (u < u_end) {
    Items it = items_of<C>(a, b);
    while (u - base >= it.units(a.kv_heads)) {
      base += it.units(a.kv_heads);
      it = items_of<C>(a, ++b);
    }
    const long long in_seq = u - base;
    const int kb0 = (int)(in_seq % it.key_blocks);
    const int item = (int)(in_seq / it.key_blocks);  // kv head, row tile
    const int rt = item % it.row_tiles, h = item / it.row_tiles;
    const int kb1 = (int)min((long long)it.key_blocks, kb0 + (u_end - u));
    const int rows_here = min(kRows, it.s.count * a.group - rt * kRows);
    const int lim0 = it.s.len - it.queries + 1;      // keys that query 0 sees
    const int qi_first = rt * kRows / a.group;
    const int qi_last = (rt * kRows + rows_here - 1) / a.group;
    const int key_end = min(min(kb1 * C::kUnit, it.s.len), lim0 + qi_last);  // keys any row of the tile sees
    const int full_end = lim0 + qi_first;            // keys that every row sees
    const int key0 = kb0 * C::kUnit;
    const int tiles = key_end > key0 ? (key_end - key0 + kTile - 1) / kTile : 0;  // of the CTA
    const int my_tiles = tiles > kw ? (tiles - kw + kKW - 1) / kKW : 0;           // of this key group

    // ---------------------------------------------------------------- loads
    // Lane l of the group's first warp holds what tile `batch0 + l` of the group needs, and issues it:
    // the rows of its pages in the cache's row list (-1: not named), and for each half of 16 keys the
    // factors of the softmax: K's scale, V's exponent, and the sum's factor 2^-(exponent + bias).
    int y0 = -1, y1 = -1, vb0 = 0, vb1 = 0, batch0 = 0;
    float ks0, ks1, ev0, ev1;
    const bool two = a.page_size == 16;  // a tile is two pages
    auto fetch = [&](int i0) {
      batch0 = i0;
      const int key = key0 + ((i0 + lane) * kKW + kw) * kTile;
      const int* row = a.page_table + (size_t)b * a.max_pages;
      auto page = [&](int at, float& ks, float& ev, int& vb) {
        ks = ev = 0.0f;
        const int id = row[at];
        if (id < 0 || id >= a.num_pages) return -1;
        const int block = id * a.kv_heads + h;
        ks = e8m0_value(a.k_scales[block]);
        vb = a.v_scales[block];
        ev = v_exponent(vb);
        return block * a.page_size;
      };
      y0 = y1 = -1;
      ks0 = ks1 = ev0 = ev1 = 0.0f;
      if (key < key_end) {
        y0 = page(key >> a.page_shift, ks0, ev0, vb0);
        y1 = y0;
        ks1 = ks0;
        ev1 = ev0;
        vb1 = vb0;
        if (two) y1 = key + 16 < key_end ? page((key >> 4) + 1, ks1, ev1, vb1) : -1;
        else if (y0 >= 0) y0 += key & (a.page_size - 1);
      }
    };
    // Issue tile i of the group into ring slot p_slot (whole warp; false on a timeout).
    auto issue = [&](int i) {
      if (i - batch0 >= 32) fetch(i);
      if constexpr (kRW > 1) {  // with one warp per group the reader itself frees the slot
        if (!mbar_wait_warp(&empty[p_slot], p_phase ^ 1)) {
          if (lane == 0) set_error(a.err, kErrReleaseTimeout);
          return false;
        }
      }
      if (lane == i - batch0) {
        meta[2 * p_slot] = make_float4(ks0, ev0, exp2f(-(float)kBias - ev0), __int_as_float((y0 >= 0) | (y1 >= 0) << 1));
        meta[2 * p_slot + 1] = make_float4(ks1, ev1, exp2f(-(float)kBias - ev1), __int_as_float(vb0 | vb1 << 8));
        uint64_t* bar = &full[p_slot];
        uint8_t* kdst = ring + p_slot * C::kStageBytes;
        const int boxes = two ? (y0 >= 0) + (y1 >= 0) : 2 * (y0 >= 0);  // of 16 rows
        mbar_arrive_expect_tx(bar, (uint32_t)(2 * boxes * 16 * kD));
#pragma unroll
        for (int half = 0; half < C::kHalves; ++half) {
          uint8_t* kd = kdst + half * (kTile * C::kBoxD);
          uint8_t* vd = kd + C::kTileBytes;
          if (y0 >= 0) {
            tma_load_2d(kd, &tm_k, bar, half * C::kBoxD, y0);
            tma_load_2d(vd, &tm_v, bar, half * C::kBoxD, y0);
          }
          if (two && y1 >= 0) {
            tma_load_2d(kd + 16 * C::kBoxD, &tm_k, bar, half * C::kBoxD, y1);
            tma_load_2d(vd + 16 * C::kBoxD, &tm_v, bar, half * C::kBoxD, y1);
          }
        }
      }
      __syncwarp();
      if (++p_slot == kStages) {
        p_slot = 0;
        p_phase ^= 1;
      }
      return true;
    };

    bool ok = true;
    if (rw == 0) {
      fetch(0);
      for (int i = 0; i < min(my_tiles, kStages) && ok; ++i) ok = issue(i);
    }

    // ---------------------------------------------------------------- Q
    // Row r: query qi = r / G, head h * G + r % G.  Each row is scaled by a power of two so that its
    // largest magnitude lies in [2^14, 2^15), then rounded to f16 and stored in fragment order:
    // per (16-row tile, step of 16 head dims) 32 lanes x {row g lo, row g + 8 lo, row g hi, row g + 8 hi}.
    for (int r = warp; r < kRows; r += C::kThreads / 32) {
      constexpr int kPer = kD / 32;
      float v[kPer];
      float amax = 0.0f;
      const bool live = r < rows_here;
      if (live) {
        const int rr = rt * kRows + r;
        const size_t row = (size_t)(it.s.begin + rr / a.group);
        const size_t at = row * (size_t)a.ldq + (size_t)(h * a.group + rr % a.group) * kD + lane * kPer;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (q_bf16)
            v[i] = __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.Q)[at + i] << 16);
          else
            v[i] = static_cast<const float*>(a.Q)[at + i];
          const float m = fabsf(v[i]);
          amax = m <= 3.402823466e38f ? fmaxf(amax, m) : amax;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = 0.0f;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = max((int)(__float_as_uint(amax) >> 23) - 127 - 14, -126);  // amax * 2^-e in [2^14, 2^15)
      const float f = copysignf(e8m0_value((uint32_t)(127 - e)), a.scale_log2);  // the scores' factor stays positive
      if (lane == 0) s_rf[r] = fabsf(a.scale_log2) * e8m0_value((uint32_t)(127 + e));
      uint16_t* dst = reinterpret_cast<uint16_t*>(s_q) + (size_t)(r >> 4) * (16 * kD);
      const int hi_row = (r >> 3) & 1, gg = r & 7;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        // head dim -> (16-byte chunk c of the K row, byte in it): lane (c >> 1) & 3 or c & 3, step, register.
        const int d = lane * kPer + i;
        const int half = d / C::kBoxD, c = (d % C::kBoxD) >> 4, within = d & 15;
        const int tt = C::kBoxD == 128 ? c >> 1 : c;
        const int step = (half * (C::kBoxD / 64) + (C::kBoxD == 128 ? (c & 1) : 0)) * 4 + (within >> 2);
        const int reg = ((within >> 1) & 1) * 2 + hi_row;
        const uint32_t pk = pack_f16x2(v[i] * f, 0.0f);
        dst[(size_t)step * 256 + (gg * 4 + tt) * 8 + reg * 2 + (within & 1)] = (uint16_t)pk;
      }
    }
    __syncthreads();

    // ---------------------------------------------------------------- tiles
    float o[kMT][kD / 8][4];
    float m[kMT][2], l[kMT][2], rf[kMT][2];
    int lim[kMT][2];
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
      for (int n = 0; n < kD / 8; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = rw * C::kRowsPerWarp + mt * 16 + g + 8 * i;
        m[mt][i] = -INFINITY;
        l[mt][i] = 0.0f;
        rf[mt][i] = s_rf[r];
        lim[mt][i] = min(lim0 + (rt * kRows + r) / a.group, it.s.len);
      }
    }
    for (int i = 0; i < my_tiles && ok; ++i) {
      if (!mbar_wait_warp(&full[c_slot], c_phase)) {
        if (lane == 0) set_error(a.err, kErrDataTimeout);
        ok = false;
        break;
      }
      const uint8_t* kt = ring + c_slot * C::kStageBytes;
      const uint8_t* vt = kt + C::kTileBytes;
      const float4 h0 = meta[2 * c_slot], h1 = meta[2 * c_slot + 1];
      const uint32_t named = __float_as_uint(h0.w);
      const int key = key0 + (i * kKW + kw) * kTile;
      const bool whole = key + kTile <= full_end && named == 3u;  // nothing of the tile is masked

      // Scores: four 8-key columns.
      float s[kMT][4][4];
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int n = 0; n < 4; ++n) s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.0f;
#pragma unroll
      for (int c = 0; c < kD / 64; ++c) {  // 64 head dims: 16 bytes per lane
        uint4 kq[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const int row = n * 8 + g;
          if constexpr (C::kBoxD == 128) {
            const int half = c >> 1, chunk = 2 * t + (c & 1);
            kq[n] = *reinterpret_cast<const uint4*>(kt + half * (kTile * 128) + row * 128 + ((chunk ^ (row & 7)) << 4));
          } else {
            kq[n] = *reinterpret_cast<const uint4*>(kt + row * 64 + ((t ^ ((row >> 1) & 3)) << 4));
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t qa[kMT][4];
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            const uint4 q = *reinterpret_cast<const uint4*>(s_q + (size_t)(rw * kMT + mt) * (16 * kD * 2) +
                                                            (c * 4 + j) * 512 + lane * 16);
            qa[mt][0] = q.x;
            qa[mt][1] = q.y;
            qa[mt][2] = q.z;
            qa[mt][3] = q.w;
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const uint32_t w = j == 0 ? kq[n].x : j == 1 ? kq[n].y : j == 2 ? kq[n].z : kq[n].w;
            uint32_t b0, b1;
            widen4(w, b0, b1);
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) mma_f16(s[mt][n], qa[mt], b0, b1);
          }
        }
      }

      // Softmax.  Keys of column n: key + 8 n + 2 t + {0, 1}; n < 2 belong to the tile's first half.
      // The maximum is taken of the raw scores, whose factor is positive.
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        uint32_t masked[2] = {0u, 0u};
        if (!whole) {
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (key + 8 * n + 2 * t + e >= lim[mt][i2] || !((named >> (n >> 1)) & 1u)) {
                  masked[i2] |= 1u << (2 * n + e);
                  s[mt][n][2 * i2 + e] = -INFINITY;
                }
        }
        float m_new[2];
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          float mx0 = max3(fmaxf(s[mt][0][2 * i2], s[mt][0][2 * i2 + 1]), s[mt][1][2 * i2], s[mt][1][2 * i2 + 1]);
          float mx1 = max3(fmaxf(s[mt][2][2 * i2], s[mt][2][2 * i2 + 1]), s[mt][3][2 * i2], s[mt][3][2 * i2 + 1]);
          float mx = fmaxf(fmaf(mx0, rf[mt][i2] * h0.x, h0.y), fmaf(mx1, rf[mt][i2] * h1.x, h1.y));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          m_new[i2] = max3(m[mt][i2], mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        }
        if (__any_sync(0xffffffffu, m_new[0] > m[mt][0] || m_new[1] > m[mt][1])) {
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2) {
            const float alpha = m_new[i2] > m[mt][i2] ? ex2(m[mt][i2] - m_new[i2]) : 1.0f;
            m[mt][i2] = m_new[i2];
            l[mt][i2] *= alpha;
#pragma unroll
            for (int n = 0; n < kD / 8; ++n) {
              o[mt][n][2 * i2] *= alpha;
              o[mt][n][2 * i2 + 1] *= alpha;
            }
          }
        }
#pragma unroll
        for (int i2 = 0; i2 < 2; ++i2) {
          const float base = m[mt][i2] == -INFINITY ? 0.0f : m[mt][i2] - (float)kBias;
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float4 hh = n < 2 ? h0 : h1;
              float p = ex2(fmaf(s[mt][n][2 * i2 + e], rf[mt][i2] * hh.x, hh.y - base));
              if (!whole && ((masked[i2] >> (2 * n + e)) & 1u)) p = 0.0f;
              s[mt][n][2 * i2 + e] = p;
              l[mt][i2] = fmaf(p, hh.z, l[mt][i2]);
            }
        }
      }

      // o += P V, 16 keys at a time.
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (!((named >> ks) & 1u)) continue;
        if ((ks == 0 ? h0.y : h1.y) == (float)kMinExp) {
          const int vb = (__float_as_int(h1.w) >> (8 * ks)) & 255;
          const float f = e8m0_value((uint32_t)(vb - kMinExp));
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[mt][2 * ks][e] *= f;
              s[mt][2 * ks + 1][e] *= f;
            }
        }
        uint32_t pa[kMT][4];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
          pa[mt][0] = pack_f16x2(s[mt][2 * ks][0], s[mt][2 * ks][1]);
          pa[mt][1] = pack_f16x2(s[mt][2 * ks][2], s[mt][2 * ks][3]);
          pa[mt][2] = pack_f16x2(s[mt][2 * ks + 1][0], s[mt][2 * ks + 1][1]);
          pa[mt][3] = pack_f16x2(s[mt][2 * ks + 1][2], s[mt][2 * ks + 1][3]);
        }
        // Keys behind the sequence hold anything, NaN too: their bytes count as zero.
        const int rk = 16 * ks + 2 * t;  // this lane's keys: rk, rk + 1, rk + 8, rk + 9
        const bool z0 = key + rk >= it.s.len, z1 = key + rk + 1 >= it.s.len;
        const bool z2 = key + rk + 8 >= it.s.len, z3 = key + rk + 9 >= it.s.len;
        uint32_t nans = 0;  // NaN codes of a tile that some rows see only in part
#pragma unroll
        for (int dg = 0; dg < kD / 32; ++dg) {
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int row = rk + (q & 1) + (q >> 1) * 8;
            if constexpr (C::kBoxD == 128) {
              const int half = dg >> 2, chunk = (dg & 3) * 2 + (g >> 2);
              w[q] = lds32(vt + half * (kTile * 128) + row * 128 + ((chunk ^ (row & 7)) << 4) + (g & 3) * 4);
            } else {
              const int chunk = dg * 2 + (g >> 2);
              w[q] = lds32(vt + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4) + (g & 3) * 4);
            }
          }
          if (!whole) {
            w[0] = z0 ? 0u : w[0];
            w[1] = z1 ? 0u : w[1];
            w[2] = z2 ? 0u : w[2];
            w[3] = z3 ? 0u : w[3];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t bad = nan_bytes(w[q]);
              nans |= bad;
              w[q] &= ~((bad >> 7) * 255u);
            }
          }
          // Pairs of keys per head dim: {k0 d0, k1 d0, k0 d1, k1 d1}, {.. d2, .. d3} and the same of k2, k3.
          const uint32_t lo01 = __byte_perm(w[0], w[1], 0x5140), lo23 = __byte_perm(w[0], w[1], 0x7362);
          const uint32_t hi01 = __byte_perm(w[2], w[3], 0x5140), hi23 = __byte_perm(w[2], w[3], 0x7362);
          uint32_t b0[4], b1[4];
          widen4(lo01, b0[0], b0[1]);
          widen4(lo23, b0[2], b0[3]);
          widen4(hi01, b1[0], b1[1]);
          widen4(hi23, b1[2], b1[3]);
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) mma_f16(o[mt][dg * 4 + q], pa[mt], b0[q], b1[q]);
        }
        // A NaN times a masked probability's zero would reach rows that do not see its token, so such
        // codes went in as zeros; the rows that see them get their NaN here.
        if (__any_sync(0xffffffffu, nans != 0)) {
          for (int kk = 0; kk < 16; ++kk) {
            const int row = 16 * ks + kk;
            if (key + row >= it.s.len) break;
#pragma unroll
            for (int dg = 0; dg < kD / 32; ++dg) {
              uint2 w;  // head dims 32 dg + 8 t ..
              if constexpr (C::kBoxD == 128) {
                const int half = dg >> 2, chunk = (dg & 3) * 2 + (t >> 1);
                w = *reinterpret_cast<const uint2*>(vt + half * (kTile * 128) + row * 128 + ((chunk ^ (row & 7)) << 4) +
                                                    (t & 1) * 8);
              } else {
                const int chunk = dg * 2 + (t >> 1);
                w = *reinterpret_cast<const uint2*>(vt + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4) + (t & 1) * 8);
              }
              const uint32_t n0 = nan_bytes(w.x), n1 = nan_bytes(w.y);
#pragma unroll
              for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    const bool seen = key + row < lim[mt][i2];
                    if (seen && ((n0 >> (8 * q + 7)) & 1u)) o[mt][dg * 4 + q][2 * i2] = __uint_as_float(0x7FC00000u);
                    if (seen && ((n1 >> (8 * q + 7)) & 1u)) o[mt][dg * 4 + q][2 * i2 + 1] = __uint_as_float(0x7FC00000u);
                  }
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[c_slot]);
      if (++c_slot == kStages) {
        c_slot = 0;
        c_phase ^= 1;
      }
      if (rw == 0 && i + kStages < my_tiles) ok = issue(i + kStages);
    }

    // ---------------------------------------------------------------- join the key groups
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[mt][i] += __shfl_xor_sync(0xffffffffu, l[mt][i], 1);
        l[mt][i] += __shfl_xor_sync(0xffffffffu, l[mt][i], 2);
        const int r = rw * C::kRowsPerWarp + mt * 16 + g + 8 * i;
        if (t == 0) {
          s_m[kw * kRows + r] = m[mt][i];
          s_l[kw * kRows + r] = l[mt][i];
        }
      }
    __syncthreads();  // every tile has been read: the ring's memory is free
    float* merge = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = rw * C::kRowsPerWarp + mt * 16 + g + 8 * i;
        float mx = s_m[r];
#pragma unroll
        for (int k = 1; k < kKW; ++k) mx = fmaxf(mx, s_m[k * kRows + r]);
        const float w = mx == -INFINITY ? 1.0f : exp2f(m[mt][i] - mx);
        float* dst = merge + (size_t)(kw * kRows + r) * C::kPitch + 8 * t;
#pragma unroll
        for (int dg = 0; dg < kD / 32; ++dg) {
          // columns 2 t and 2 t + 1 of the four products: head dims 32 dg + 8 t + {0 .. 3}, {4 .. 7}
          float4 lo, hi;
          lo.x = o[mt][dg * 4 + 0][2 * i] * w;
          lo.y = o[mt][dg * 4 + 1][2 * i] * w;
          lo.z = o[mt][dg * 4 + 2][2 * i] * w;
          lo.w = o[mt][dg * 4 + 3][2 * i] * w;
          hi.x = o[mt][dg * 4 + 0][2 * i + 1] * w;
          hi.y = o[mt][dg * 4 + 1][2 * i + 1] * w;
          hi.z = o[mt][dg * 4 + 2][2 * i + 1] * w;
          hi.w = o[mt][dg * 4 + 3][2 * i + 1] * w;
          *reinterpret_cast<float4*>(dst + dg * 32) = lo;
          *reinterpret_cast<float4*>(dst + dg * 32 + 4) = hi;
        }
      }
    __syncthreads();
    const bool complete = kb0 == 0 && kb1 == it.key_blocks;
    const int slot = 2 * blockIdx.x + (u == u_begin ? 0 : 1);
    constexpr int kQuads = kD / 4;
    for (int x = tid; x < rows_here * kQuads; x += C::kThreads) {
      const int r = x / kQuads, d = (x % kQuads) * 4;
      float mx = s_m[r];
#pragma unroll
      for (int k = 1; k < kKW; ++k) mx = fmaxf(mx, s_m[k * kRows + r]);
      float sum = 0.0f;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kKW; ++k) {
        sum += s_l[k * kRows + r] * (mx == -INFINITY ? 1.0f : exp2f(s_m[k * kRows + r] - mx));
        const float4 v = *reinterpret_cast<const float4*>(merge + (size_t)(k * kRows + r) * C::kPitch + d);
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      if (complete) {
        const float inv = sum == 0.0f ? 0.0f : kUnbias / sum;  // a row that sees nothing: zeros
        const int rr = rt * kRows + r;
        const size_t row = (size_t)(it.s.begin + rr / a.group);
        const int head = h * a.group + rr % a.group;
        const size_t at = row * (size_t)a.ldo + (size_t)head * kD + d;
        if (a.out_bf16)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
              make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) =
              make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (a.lse && d == 0) a.lse[row * a.q_heads + head] = sum == 0.0f ? -INFINITY : kLn2 * (mx + log2f(sum));
      } else {
        *reinterpret_cast<float4*>(a.partial + ((size_t)slot * kRows + r) * kD + d) = acc;
        if (d == 0) {
          float* ml = a.partial + (size_t)2 * a.runs * kRows * kD;
          ml[(size_t)slot * kRows + r] = mx;
          ml[(size_t)(2 * a.runs + slot) * kRows + r] = sum;
        }
      }
    }
    // The ring's memory was written by ordinary stores; the next item's copies come through the
    // asynchronous proxy.
    fence_proxy_async_smem();
    __syncthreads();
    u += kb1 - kb0;
  }
}

// Joins the partials of the items cut by run borders, in key order.  One warp per row: a lane weighs
// every 32nd partial, then the lanes take the head dims and add all partials in order.
// blockIdx.x: kv head and group of kJoinRows rows of the item list; y: sequence.
constexpr int kJoinRows = 4;
template <class C>
__global__ void __launch_bounds__(32 * kJoinRows) k_attn_kv8_join(const AttnArgs a, const int groups) {
  constexpr int kD = C::kD, kRows = C::kRows, kPer = kD / 32;
  __shared__ float s_w[kJoinRows][64];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y, h = blockIdx.x / groups, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rr = (blockIdx.x % groups) * kJoinRows + warp;  // row of the (sequence, kv head)
  const Items it = items_of<C>(a, b);
  const int rt = rr / kRows, r = rr % kRows;
  if (rr >= it.s.count * a.group) return;
  long long W = 0, base = 0;
  for (int q = lane; q < a.batch; q += 32) {
    const long long n = items_of<C>(a, q).units(a.kv_heads);
    W += n;
    base += q < b ? n : 0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    W += __shfl_xor_sync(0xffffffffu, W, o);
    base += __shfl_xor_sync(0xffffffffu, base, o);
  }
  const int runs = runs_used(W, a.runs, a.min_units);
  const long long u0 = base + (long long)(h * it.row_tiles + rt) * it.key_blocks, u1 = u0 + it.key_blocks;
  // Run of unit u: the last r with W r / runs <= u.
  auto run_of = [&](long long u) {
    int q = (int)((u * runs) / W);
    while (W * (q + 1) / runs <= u) ++q;
    while (W * q / runs > u) --q;
    return q;
  };
  const int r0 = run_of(u0), r1 = run_of(u1 - 1);
  if (r0 == r1) return;  // written by its CTA
  const int slot0 = 2 * r0 + (W * r0 / runs == u0 ? 0 : 1);
  const float* ml = a.partial + (size_t)2 * a.runs * kRows * kD;
  const float* ll = ml + (size_t)2 * a.runs * kRows;
  auto at = [&](int c) { return (size_t)(c == r0 ? slot0 : 2 * c) * kRows + r; };
  float mx = -INFINITY;
  for (int c = r0 + lane; c <= r1; c += 32) mx = fmaxf(mx, ml[at(c)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.0f, acc[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
  for (int c0 = r0; c0 <= r1; c0 += 64) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = c0 + 32 * j + lane;
      float w = 0.0f;
      if (c <= r1) {
        w = mx == -INFINITY ? 1.0f : exp2f(ml[at(c)] - mx);
        sum += w * ll[at(c)];
      }
      s_w[warp][32 * j + lane] = w;
    }
    __syncwarp();
    const int n = min(64, r1 - c0 + 1);
#pragma unroll 8
    for (int c = 0; c < n; ++c) {
      const float w = s_w[warp][c];
      const float* src = a.partial + at(c0 + c) * kD + lane * kPer;
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        const float2 v = *reinterpret_cast<const float2*>(src + i);
        acc[i] = fmaf(w, v.x, acc[i]);
        acc[i + 1] = fmaf(w, v.y, acc[i + 1]);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = sum == 0.0f ? 0.0f : kUnbias / sum;  // a row that sees nothing: zeros
  const size_t row = (size_t)(it.s.begin + rr / a.group);
  const int head = h * a.group + rr % a.group;
  const size_t o = row * (size_t)a.ldo + (size_t)head * kD + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {
    if (a.out_bf16)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + o + i) = pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
    else
      *reinterpret_cast<float2*>(static_cast<float*>(a.out) + o + i) = make_float2(acc[i] * inv, acc[i + 1] * inv);
  }
  if (a.lse && lane == 0) a.lse[row * a.q_heads + head] = sum == 0.0f ? -INFINITY : kLn2 * (mx + log2f(sum));
}

constexpr int kMaxRuns = 444;  // 148 SMs x 3 CTAs

template <class C>
cudaError_t launch_cfg(const AttnKv8Launch& L, cudaStream_t stream) {
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

  auto kern = k_attn_kv8<C>;
  static int occ[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (occ[dev] == 0) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, C::kThreads, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    occ[dev] = n < 1 ? 1 : n;
  }
  const int slots = sm_count() * occ[dev];
  a.runs = slots < kMaxRuns ? slots : kMaxRuns;
  a.min_units = 1;

  CUtensorMap tm_k, tm_v;
  const uint64_t rows = (uint64_t)L.num_pages * L.kv_heads * L.page_size;
  const uint32_t box_rows = L.page_size < kTile ? L.page_size : kTile;
  const CUtensorMapSwizzle sw = C::kBoxD == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!make_map_2d(&tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.k_codes, C::kD, rows, C::kD, C::kBoxD, box_rows, sw) ||
      !make_map_2d(&tm_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.v_codes, C::kD, rows, C::kD, C::kBoxD, box_rows, sw))
    return cudaErrorInvalidValue;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.runs);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tm_k, tm_v, a, L.q_bf16 ? 1 : 0);
  if (e != cudaSuccess) return e;
  // No sequence can be longer than its page table: when that is one unit, no item is ever cut.
  if ((long long)L.max_pages * L.page_size <= C::kUnit) return cudaSuccess;
  const long long groups = ((long long)L.max_q_len * a.group + kJoinRows - 1) / kJoinRows;
  if (groups * L.kv_heads >= (1LL << 31)) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3((unsigned)(groups * L.kv_heads), (unsigned)L.batch);
  cfg.blockDim = dim3(32 * kJoinRows);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, k_attn_kv8_join<C>, a, (int)groups);
}

// Rows of an item by the most rows a sequence can have (queries times heads per kv head).
template <int kD>
cudaError_t launch_rows(const AttnKv8Launch& L, cudaStream_t stream) {
  const long long rows = (long long)L.max_q_len * (L.q_heads / L.kv_heads);
  constexpr bool kWide = kD == 256;  // two 16-row tiles per warp would not fit its registers
  if (rows <= 16) return launch_cfg<AttnCfg<kD, 1, 1, 4, kD == 64 ? 4 : 2, kWide ? 1 : 3>>(L, stream);
  if (rows <= 32) return launch_cfg<AttnCfg<kD, kWide ? 1 : 2, kWide ? 2 : 1, 4, kD == 64 ? 4 : 2, kWide ? 1 : 2>>(L, stream);
  return launch_cfg<AttnCfg<kD, kWide ? 1 : 2, kWide ? 4 : 2, 2, kD == 64 ? 4 : 3, kWide ? 1 : 2>>(L, stream);
}

int rows_per_item(long long rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

}  // namespace

size_t attn_kv8_workspace_bytes(int max_q_len, int q_heads, int kv_heads, int head_dim) {
  const size_t rows = (size_t)rows_per_item((long long)max_q_len * (q_heads / kv_heads));
  return 2 * (size_t)kMaxRuns * rows * ((size_t)head_dim + 2) * sizeof(float);
}

cudaError_t launch_attn_kv8(const AttnKv8Launch& L, cudaStream_t stream) {
  switch (L.head_dim) {
    case 64: return launch_rows<64>(L, stream);
    case 128: return launch_rows<128>(L, stream);
    case 256: return launch_rows<256>(L, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace batq
