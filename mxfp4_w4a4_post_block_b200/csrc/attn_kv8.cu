// k_attn_kv8: attention of few queries per sequence over the 8-bit paged cache (kv8.cuh).
//
// For query i of a sequence with n queries and L tokens in the cache (the queries' own among them),
// head h of kv head j = h / G:
//   s_t = scale * 2^ek(t) * <q, K_t>,  t <= L - n + i;   p = softmax(s);   o = sum_t p_t 2^ev(t) V_t
// in one pass over the cache with a running maximum and sum (fp32) per row.
//
// The G heads of a kv head times the queries are the 8 columns, and K's and V's own dimensions the 16
// rows, of m16n8k16 matrix instructions (S^T = K Q^T, O^T = V^T P^T): a decode step has few rows, and
// with those on the 16-row side half of every instruction and accumulator would be padding.  E4M3
// widens exactly to f16, so K and V enter as f16 codes and the page scales stay outside: 2^ek
// multiplies the fp32 scores, 2^ev rides on them (below).  Q is rounded to f16 after an exact
// power-of-two normalisation of its row (bf16 queries keep all their bits down to 2^-28 of the row's
// largest; fp32 queries keep 11); probabilities are rounded to f16 (2^-11 relative), less than the
// bf16 output's own step.
//
// Layout in registers.  The reduction dimensions may be ordered freely, as long as both operands
// agree, so a lane reads 16 consecutive bytes of a K row (one LDS.128 feeds four K steps) and, of V,
// four bytes (head dims) of each of four keys, transposed by byte permutes into the f16 pairs (two
// keys of one head dim) that the instruction wants; movmatrix turns the probabilities from S^T's
// accumulator layout into the second product's operand.  Tiles of 32 keys come by TMA with the
// 128-byte (head dim 64: 64-byte) swizzle, which makes both reads conflict-free.
//
// Work split.  The keys of all (sequence, kv head, row tile) items are cut into blocks of kUnit keys;
// the list of all blocks is dealt out in equal contiguous runs, one per CTA, computed by each CTA
// from seq_lens.  A CTA whose run covers an item writes its output; items cut by run borders leave
// (m, l, o) partials in the workspace (at most two per CTA: its first and its last item), joined in
// key order by k_attn_kv8_join.  Within a CTA, kKW key groups take every kKW-th tile, each with a
// ring of its own (K and V tiles in turn), and kRW warps of a group share its tiles for further rows.
//
// What bounds it is the issue of instructions: widening K and V, the softmax's and the loads' address
// arithmetic are about 820 of them per 32 keys and 8 rows, at half of the issue slots; so head dim 128 with
// long page tables has the kernel in attn_kv8_tc.cu.  Measured: 16 sequences of up to 16000 tokens, 4 heads of
// 8 queries: 33 us at head dim 64 (2.1 TB/s), 67 us at 256 (4.2 TB/s); 3 sequences of 100 tokens 6 us, the
// launch and one tile's way through it.  More rows cost more softmax: five queries each 74 and 130 us.
#include <cstdint>
#include <type_traits>

#include "attn_kv8.cuh"

namespace batq {
namespace {

constexpr int kTile = 32;  // keys per tile
constexpr int kBias = 15;  // of the weights' exponents (below)
constexpr float kUnbias = 1.0f / (1 << kBias);

// kD: head dim; kNT: 8-row tiles per warp; kRW: row warps; kKW: key groups; kSlots: ring slots (a K or
// a V tile each) per key group; kCtas: CTAs per SM that registers and shared memory are laid out for.
template <int kD_, int kNT_, int kRW_, int kKW_, int kSlots_, int kCtas_>
struct AttnCfg {
  static constexpr int kOver = 0;
  static constexpr float kOutUnit = kUnbias;                // what the accumulators and partials count
  static constexpr int kD = kD_, kNT = kNT_, kRW = kRW_, kKW = kKW_, kSlots = kSlots_, kCtas = kCtas_;
  static constexpr int kRowsPerWarp = 8 * kNT;
  static constexpr int kRows = kRowsPerWarp * kRW;
  static constexpr int kThreads = 32 * kRW * kKW;
  static constexpr int kUnit = kTile * kKW;                 // keys per work unit
  static constexpr int kBoxD = kD < 128 ? kD : 128;         // bytes per row of one swizzled box
  static constexpr int kHalves = kD / kBoxD;                // boxes along the head dim
  static constexpr int kTileBytes = kTile * kD;
  static constexpr int kRingBytes = kKW * kSlots * kTileBytes;
  static constexpr int kPitch = kD + 4;                     // floats per row of the merge buffer
  static constexpr int kMergeBytes = kKW * kRows * kPitch * 4;
  static constexpr int kDataBytes = kRingBytes > kMergeBytes ? kRingBytes : kMergeBytes;  // the merge reuses the ring
  static constexpr int kMetas = kSlots <= 4 ? 4 : 8;         // more than the tiles whose factors are alive at a time
  static constexpr int kQBytes = kRows * kD * 2;
  static constexpr int kSmallBytes = kRows * 4 + 2 * kKW * kRows * 4 + 2 * kKW * kSlots * 8 + kKW * kMetas * 32 + 64;
  static constexpr int kSmemBytes = kDataBytes + kQBytes + kSmallBytes + 1024;
};

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

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// V's page scales ride on the scores: with x_t the score in log2 units and 2^ev(t) the scale of token
// t's V block, the weights in the matrix instruction are p_t = 2^(x_t + ev(t) - m + kBias), m the
// running maximum of x + ev, and the sum takes p_t 2^-(ev(t) + kBias) = 2^(x_t - m).  So f16 keeps 11
// bits of every weight that matters beside the row's largest product of probability and scale (the
// bias puts that one at 2^15, and f16's smallest step 2^39 below it) however far apart the blocks'
// scales are, and the accumulators need no unit of their own.  Scales below 2^kMinExp (an all-zero
// block has 2^-127) ride as 2^kMinExp, and the rest multiplies the f16 weights.  From the first tile
// on whose |ev| is beyond kSameExp, a sum has a reference of its own (kFarExp has which) and
// exponentials of its own; a piece's outputs are brought to that reference at its end.  (Up to there
// the factor 2^(m - m') of a new maximum leaves fp32's range only where the sum so far has no bits in
// the new one: -126 + 2 * 48 = -30.)
constexpr int kMinExp = -100;
constexpr float kSameExp = 48.0f;
static_assert(kSameExp <= kFarExp, "the reference so far is the sum's own");
__device__ __forceinline__ float v_exponent(int byte) {
  return byte == 255 ? __uint_as_float(0x7FC00000u) : (float)max(byte - 127, kMinExp);
}

__device__ __forceinline__ uint32_t lds32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }

// Transposes an 8 x 8 matrix of 16-bit values held one row per four lanes.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Adds the exponentials of a tile's scores to two rows' sums whose references stand at `ref` and `ref + 1`: a, b the
// scores of the halves' keys as they lie (row 0, row 1, row 0, row 1), f their factors (a's two, b's two), e_base V's
// exponents and what the scores count from, bit 4 b + i of `masked` a score that is not.  Returns the sums, where the
// references stand from what the scores count from, and their changes: the outputs' references go by those, since
// fp32 holds large scores in steps that V's exponents are lost in.
struct FarSums {
  float l[2], at[2], change[2];
};
__device__ __forceinline__ FarSums far_sums(const float4 a, const float4 b, const float4 f, const float4 e_base, const float2 l,
                                         const uint32_t masked, float* const ref) {
  const float s[2][4] = {{a.x, a.y, a.z, a.w}, {b.x, b.y, b.z, b.w}};
  const float fs[2][2] = {{f.x, f.y}, {f.z, f.w}}, base[2] = {e_base.z, e_base.w};
  float sums[2] = {l.x, l.y};
  FarSums r;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float mx = fmaxf(fmaf(fmaxf(s[0][e], s[0][2 + e]), fs[0][e], near_exponent(e_base.x)),
                     fmaf(fmaxf(s[1][e], s[1][2 + e]), fs[1][e], near_exponent(e_base.y)));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
    const float before = ref[e], top = fmaxf(before, mx + base[e]);
    if (top > before) sums[e] = times(sums[e], pow2_of(before - top));
    __syncwarp();
    if ((threadIdx.x & 28) == 0) ref[e] = top;
    __syncwarp();
    const float from = base[e] == 0.0f ? top : mx - ((mx + base[e]) - top);
    const float less = top == -INFINITY ? 0.0f : from;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int mk = q >> 1, at = 2 * (q & 1) + e;
      if (!((masked >> (4 * mk + at)) & 1u)) sums[e] += ex2(fmaf(s[mk][at], fs[mk][e], -less));
    }
    r.l[e] = sums[e];
    r.at[e] = less;
    r.change[e] = top > before ? before - top : 0.0f;
  }
  return r;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
    k_attn_kv8(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const AttnArgs a,
               const int q_bf16) {
  constexpr int kD = C::kD, kNT = C::kNT, kKW = C::kKW, kRW = C::kRW, kSlots = C::kSlots, kRows = C::kRows;
  extern __shared__ uint8_t smem_raw[];
  // (an offset, so that the compiler still knows these for shared addresses)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_q = smem + C::kDataBytes;                                       // Q fragments (f16)
  float* s_rf = reinterpret_cast<float*>(s_q + C::kQBytes);                  // [kRows] factor of each row's scores
  float* s_m = s_rf + kRows;                                                 // [kKW][kRows]
  float* s_l = s_m + kKW * kRows;                                            // [kKW][kRows]
  float4* s_meta = reinterpret_cast<float4*>(s_l + kKW * kRows);             // [kKW][kMetas][2], see fetch
  uint64_t* s_full = reinterpret_cast<uint64_t*>(s_meta + kKW * C::kMetas * 2);  // [kKW][kSlots]
  uint64_t* s_empty = s_full + kKW * kSlots;                                 // [kKW][kSlots]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kw = warp / kRW, rw = warp % kRW;
  const int g = lane >> 2, t = lane & 3;
  if (tid == 0) {
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
    for (int i = 0; i < kKW * kSlots; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kRW);
    }
    fence_barrier_init();
  }
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();

  const Runs runs = runs_of(count_units<C>(a, 0, lane).x, a.runs);
  if ((int)blockIdx.x >= runs.count) return;
  int u = runs.begin(blockIdx.x);
  const int u_begin = u, u_end = runs.begin(blockIdx.x + 1);

  // The sequence of unit u: each warp scans the batch.
  int b = 0;
  int base = 0;  // units before sequence b
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int n = b0 + lane < a.batch ? items_of<C>(a, b0 + lane).units(a.kv_heads) : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, n > 0 && base + incl > u);
    if (hit) {
      const int src = __ffs(hit) - 1;
      b = b0 + src;
      base += __shfl_sync(0xffffffffu, incl - n, src);
      break;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }

  uint8_t* ring = smem + kw * (kSlots * C::kTileBytes);
  uint64_t* full = s_full + kw * kSlots;
  uint64_t* empty = s_empty + kw * kSlots;
  float4* meta = s_meta + kw * C::kMetas * 2;
  int p_slot = 0, c_slot = 0;         // producer's and consumer's ring slots
  uint32_t p_phase = 0, c_phase = 0;

  while (u < u_end) {
    Items it = items_of<C>(a, b);
    while (u - base >= it.units(a.kv_heads)) {
      base += it.units(a.kv_heads);
      it = items_of<C>(a, ++b);
    }
    const int item = (u - base) / it.key_blocks;     // kv head, row tile
    const int kb0 = (u - base) - item * it.key_blocks;
    const int rt = item % it.row_tiles, h = item / it.row_tiles;
    const int kb1 = min(it.key_blocks, kb0 + (u_end - u));
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
    float4 f0, f1;
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
      float ks0 = 0.0f, ks1 = 0.0f, ev0 = 0.0f, ev1 = 0.0f;
      if (key < key_end) {
        y0 = page(key >> a.page_shift, ks0, ev0, vb0);
        y1 = y0;
        ks1 = ks0;
        ev1 = ev0;
        vb1 = vb0;
        if (two) y1 = key + 16 < key_end ? page((key >> 4) + 1, ks1, ev1, vb1) : -1;
        else if (y0 >= 0) y0 += key & (a.page_size - 1);
      }
      f0 = make_float4(ks0, ev0, exp2f(-(float)kBias - ev0), __int_as_float((y0 >= 0) | (y1 >= 0) << 1));
      f1 = make_float4(ks1, ev1, exp2f(-(float)kBias - ev1), __int_as_float(vb0 | vb1 << 8));
    };
    // Issue load j of the group (tile j / 2: K, then V) into ring slot p_slot (whole warp; false on a timeout).
    auto issue = [&](int j) {
      const int i = j >> 1;
      if (i - batch0 >= 32) fetch(i);
      if constexpr (kRW > 1) {  // with one warp per group the reader itself frees the slot
        if (!mbar_wait_warp(&empty[p_slot], p_phase ^ 1)) {
          if (lane == 0) set_error(a.err, kErrReleaseTimeout);
          return false;
        }
      }
      if (lane == i - batch0) {
        uint64_t* bar = &full[p_slot];
        uint8_t* dst = ring + p_slot * C::kTileBytes;
        const CUtensorMap* map = (j & 1) ? &tm_v : &tm_k;
        if (!(j & 1)) {
          meta[2 * (i % C::kMetas)] = f0;
          meta[2 * (i % C::kMetas) + 1] = f1;
        }
        const int boxes = two ? (y0 >= 0) + (y1 >= 0) : 2 * (y0 >= 0);  // of 16 rows
        mbar_arrive_expect_tx(bar, (uint32_t)(boxes * 16 * kD));
#pragma unroll
        for (int half = 0; half < C::kHalves; ++half) {
          uint8_t* d = dst + half * (kTile * C::kBoxD);
          if (y0 >= 0) tma_load_2d(d, map, bar, half * C::kBoxD, y0);
          if (two && y1 >= 0) tma_load_2d(d + 16 * C::kBoxD, map, bar, half * C::kBoxD, y1);
        }
      }
      __syncwarp();
      if (++p_slot == kSlots) {
        p_slot = 0;
        p_phase ^= 1;
      }
      return true;
    };

    bool ok = true;
    const int loads = 2 * my_tiles;
    if (rw == 0) {
      fetch(0);
      for (int j = 0; j < min(loads, kSlots) && ok; ++j) ok = issue(j);
    }
    // The slot just read is free: load j + kSlots goes there.
    auto release = [&](int j) {
      __syncwarp();
      if constexpr (kRW > 1) {
        if (lane == 0) mbar_arrive(&empty[c_slot]);
      }
      if (++c_slot == kSlots) {
        c_slot = 0;
        c_phase ^= 1;
      }
      if (rw == 0 && j + kSlots < loads) ok = issue(j + kSlots);
    };

    // ---------------------------------------------------------------- Q
    // Row r: query qi = r / G, head h * G + r % G.  Each row is scaled by a power of two so that its
    // largest magnitude lies in [2^14, 2^15), then rounded to f16 and stored in fragment order:
    // per (8-row tile, step of 16 head dims) 32 lanes x {row g lo, row g hi}.
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
        for (int i = 0; i < kPer; i += 2) {
          if (q_bf16) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.Q) + at + i);
            v[i] = __uint_as_float(w << 16);
            v[i + 1] = __uint_as_float(w & 0xFFFF0000u);
          } else {
            const float2 w = *reinterpret_cast<const float2*>(static_cast<const float*>(a.Q) + at + i);
            v[i] = w.x;
            v[i + 1] = w.y;
          }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const float m = fabsf(v[i]);
          amax = m <= 3.402823466e38f ? fmaxf(amax, m) : amax;
          v[i] = m <= 3.402823466e38f ? v[i] : __uint_as_float(0x7FC00000u);  // (infinite scores could sum to nothing)
        }
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[i] = 0.0f;
      }
      amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));  // not negative: ordered as bits
      const int e = max((int)(__float_as_uint(amax) >> 23) - 127 - 14, -126);  // amax * 2^-e in [2^14, 2^15)
      const float f = copysignf(e8m0_value((uint32_t)(127 - e)), a.scale_log2);  // the scores' factor stays positive
      if (lane == 0) s_rf[r] = fabsf(a.scale_log2) * e8m0_value((uint32_t)(127 + e));
      uint8_t* dst = s_q + (size_t)(r >> 3) * (8 * kD * 2);
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        // head dim -> 16-byte chunk c of the K row and the byte in it: lane c >> 1 (c for 64-byte rows), step, register
        const int d = lane * kPer + i;
        const int half = d / C::kBoxD, c = (d % C::kBoxD) >> 4, within = d & 15;
        const int tt = C::kBoxD == 128 ? c >> 1 : c;
        const int step = (half * (C::kBoxD / 64) + (C::kBoxD == 128 ? (c & 1) : 0)) * 4 + (within >> 2);
        *reinterpret_cast<uint32_t*>(dst + step * 256 + ((r & 7) * 4 + tt) * 8 + ((within >> 1) & 1) * 4) =
            pack_f16x2(v[i] * f, v[i + 1] * f);
      }
    }
    __syncthreads();

    // ---------------------------------------------------------------- tiles
    // This lane's rows: 8 n + 2 t and the next of its warp's; keys of a tile: 16 mk + g and + 8.
    float o[kD / 16][kNT][4];
    float m[kNT][2], l[kNT][2], rf[kNT][2];
    bool far = false;  // the sums have references of their own (the same for the warp), in s_m, and m counts from them
    int lim[kNT][2];
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
#pragma unroll
      for (int d = 0; d < kD / 16; ++d) o[d][n][0] = o[d][n][1] = o[d][n][2] = o[d][n][3] = 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = rw * C::kRowsPerWarp + n * 8 + 2 * t + i;
        m[n][i] = -INFINITY;
        l[n][i] = 0.0f;
        rf[n][i] = s_rf[r];
        lim[n][i] = min(lim0 + (rt * kRows + r) / a.group, it.s.len);
      }
    }
    // Places in a swizzled tile, head dim chunks XORed with the row: the 16 bytes (2 t; 64-byte rows: t) of
    // key g, and the four bytes 4 g .. of keys 2 t and 2 t + 1.  Rows 8 further have the same pattern.
    uint32_t k_at, v_at[2];
    if constexpr (C::kBoxD == 128) {
      k_at = g * 128 + (((2 * t) ^ g) << 4);
#pragma unroll
      for (int q = 0; q < 2; ++q) v_at[q] = (2 * t + q) * 128 + (((g >> 2) ^ (2 * t + q)) << 4) + (g & 3) * 4;
    } else {
      k_at = g * 64 + ((t ^ ((g >> 1) & 3)) << 4);
#pragma unroll
      for (int q = 0; q < 2; ++q) v_at[q] = (2 * t + q) * 64 + (((g >> 2) ^ t) << 4) + (g & 3) * 4;
    }
    const uint8_t* my_q = s_q + rw * (C::kRowsPerWarp * kD * 2) + lane * 8;
    auto landed = [&]() {
      if (mbar_wait_warp(&full[c_slot], c_phase)) return true;
      if (lane == 0) set_error(a.err, kErrDataTimeout);
      return ok = false;
    };
    // Tile i, whose K has landed.  kWhole: nothing of it is masked (all but a sequence's last tiles); kFar: `far`.
    auto tile = [&](auto whole_tag, auto far_tag, const int i, const int key, const float4 h0, const float4 h1) {
      constexpr bool kWhole = decltype(whole_tag)::value, kFar = decltype(far_tag)::value;
      const uint32_t named = kWhole ? 3u : __float_as_uint(h0.w);

      // S^T: two 16-key tiles by the warp's rows.
      float s[2][kNT][4];
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int mk = 0; mk < 2; ++mk) s[mk][n][0] = s[mk][n][1] = s[mk][n][2] = s[mk][n][3] = 0.0f;
      {
        const uint8_t* kt = ring + c_slot * C::kTileBytes;
#pragma unroll
        for (int c = 0; c < kD / 64; ++c) {  // 64 head dims: 16 bytes per lane and key
          uint4 kq[4];
#pragma unroll
          for (int n = 0; n < 4; ++n)
            kq[n] = *reinterpret_cast<const uint4*>(kt + (k_at ^ ((c & 1) << 4)) + (c >> 1) * (kTile * 128) +
                                                    n * (8 * C::kBoxD));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint2 q[kNT];
#pragma unroll
            for (int n = 0; n < kNT; ++n)
              q[n] = *reinterpret_cast<const uint2*>(my_q + n * (8 * kD * 2) + (c * 4 + j) * 256);
#pragma unroll
            for (int mk = 0; mk < 2; ++mk) {
              uint32_t ka[4];
              const uint4 k0 = kq[2 * mk], k1 = kq[2 * mk + 1];
              widen4(j == 0 ? k0.x : j == 1 ? k0.y : j == 2 ? k0.z : k0.w, ka[0], ka[2]);
              widen4(j == 0 ? k1.x : j == 1 ? k1.y : j == 2 ? k1.z : k1.w, ka[1], ka[3]);
#pragma unroll
              for (int n = 0; n < kNT; ++n) mma_f16(s[mk][n], ka, q[n].x, q[n].y);
            }
          }
        }
      }
      release(2 * i);

      // Softmax.  The maximum is taken of the raw scores, whose factor is positive.
      uint32_t pb[2][kNT][2];  // P^T: the second product's operand
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        uint32_t masked = 0;
        if constexpr (!kWhole) {
#pragma unroll
          for (int mk = 0; mk < 2; ++mk)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key + 16 * mk + g + 8 * (e >> 1) >= lim[n][e & 1] || !((named >> mk) & 1u)) {
                masked |= 1u << (4 * mk + e);
                s[mk][n][e] = -INFINITY;
              }
        }
        float f0[2], f1[2], base[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f0[e] = rf[n][e] * h0.x;
          f1[e] = rf[n][e] * h1.x;
          base[e] = 0.0f;
        }
        // The maximum is taken of rounded scores, the weights' differences of exact ones: so scores that may pass
        // 2^21 (the products' sums stay below 2^32) are rounded first, and counted from the tile's largest.
        if (__any_sync(0xffffffffu, fmaxf(fmaxf(f0[0], f0[1]), fmaxf(f1[0], f1[1])) > 0x1p-11f)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int q = 0; q < 4; q += 2) {  // (one factor after the other: their product may leave fp32's range)
#pragma unroll
              for (int mk = 0; mk < 2; ++mk) {
                const float f = mk == 0 ? h0.x : h1.x;
                float& v = s[mk][n][q + e];
                if (v != -INFINITY) v = f < 1.0f ? v * f * rf[n][e] : v * rf[n][e] * f;
              }
            }
            float mx = fmaxf(fmaxf(s[0][n][e], s[0][n][2 + e]), fmaxf(s[1][n][e], s[1][n][2 + e]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            base[e] = mx > -INFINITY ? mx : 0.0f;
#pragma unroll
            for (int q = 0; q < 4; q += 2) {
              s[0][n][q + e] -= base[e];
              s[1][n][q + e] -= base[e];
            }
            f0[e] = f1[e] = 1.0f;
          }
        }
        float m_new[2], local[2];
        if constexpr (kFar) {
          const FarSums r =
              far_sums(make_float4(s[0][n][0], s[0][n][1], s[0][n][2], s[0][n][3]),
                       make_float4(s[1][n][0], s[1][n][1], s[1][n][2], s[1][n][3]), make_float4(f0[0], f0[1], f1[0], f1[1]),
                       make_float4(h0.y, h1.y, base[0], base[1]), make_float2(l[n][0], l[n][1]), masked,
                       s_m + kw * kRows + rw * C::kRowsPerWarp + n * 8 + 2 * t);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[n][e] = r.l[e];
            m[n][e] += r.change[e];
            base[e] = -r.at[e];  // (m counts from there)
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x0 = fmaf(fmaxf(s[0][n][e], s[0][n][2 + e]), f0[e], h0.y);
          const float x1 = fmaf(fmaxf(s[1][n][e], s[1][n][2 + e]), f1[e], h1.y);
          float mx = fmaxf(x0, x1);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          local[e] = mx;
          m_new[e] = fmaxf(m[n][e], mx + base[e]);
        }
        if (__any_sync(0xffffffffu, m_new[0] > m[n][0] || m_new[1] > m[n][1])) {
          float alpha[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            alpha[e] = m_new[e] > m[n][e] ? ex2(m[n][e] - m_new[e]) : 1.0f;
            m[n][e] = m_new[e];
            if (!kFar) l[n][e] *= alpha[e];
          }
#pragma unroll
          for (int d = 0; d < kD / 16; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][n][e] *= alpha[e & 1];
        }
        float b0[2], b1[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          // -m + kBias for scores counted from `base`.
          const float from = base[e] == 0.0f ? m[n][e] : local[e] - ((local[e] + base[e]) - m[n][e]);
          const float less = m[n][e] == -INFINITY ? 0.0f : from - (float)kBias;
          b0[e] = h0.y - less;
          b1[e] = h1.y - less;
        }
#pragma unroll
        for (int mk = 0; mk < 2; ++mk) {
          const float4 hh = mk == 0 ? h0 : h1;
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2(fmaf(s[mk][n][e], mk == 0 ? f0[e & 1] : f1[e & 1], mk == 0 ? b0[e & 1] : b1[e & 1]));
            if (!kWhole && ((masked >> (4 * mk + e)) & 1u))
              p[e] = 0.0f;  // (a NaN scale is not for this row's sum either)
            else if (!kFar)
              l[n][e & 1] = fmaf(p[e], hh.z, l[n][e & 1]);
          }
          if (hh.y == (float)kMinExp) {
            const float f = e8m0_value((uint32_t)(((__float_as_int(h1.w) >> (8 * mk)) & 255) - kMinExp));
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] *= f;
          }
          pb[mk][n][0] = transpose8x8(pack_f16x2(p[0], p[1]));
          pb[mk][n][1] = transpose8x8(pack_f16x2(p[2], p[3]));
        }
      }

      // O^T += V^T P^T, 16 keys at a time.
      if (!landed()) return;
      const uint8_t* vt = ring + c_slot * C::kTileBytes;
      // Four head dims (4 g ..) of the 32-dim group dg of any key of this tile.
      auto v_word = [&](int row, int dg) {
        if constexpr (C::kBoxD == 128) {
          const int half = dg >> 2, chunk = (dg & 3) * 2 + (g >> 2);
          return lds32(vt + half * (kTile * 128) + row * 128 + ((chunk ^ (row & 7)) << 4) + (g & 3) * 4);
        } else {
          const int chunk = dg * 2 + (g >> 2);
          return lds32(vt + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4) + (g & 3) * 4);
        }
      };
#pragma unroll
      for (int mk = 0; mk < 2; ++mk) {
        if (!((named >> mk) & 1u)) continue;
        const int rk = 16 * mk + 2 * t;  // this lane's keys: rk, rk + 1, rk + 8, rk + 9
        uint32_t nans = 0;               // NaN codes of a tile that some rows see only in part
#pragma unroll
        for (int dg = 0; dg < kD / 32; ++dg) {
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            w[q] = lds32(vt + (v_at[q & 1] ^ ((dg & 3) << 5)) + (dg >> 2) * (kTile * 128) +
                         (16 * mk + 8 * (q >> 1)) * C::kBoxD);
          if constexpr (!kWhole) {
            // Keys behind the sequence hold anything, NaN too: their bytes count as zero.
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (key + rk + (q & 1) + (q >> 1) * 8 >= it.s.len) w[q] = 0u;
              const uint32_t bad = nan_bytes(w[q]);
              nans |= bad;
              w[q] &= ~((bad >> 7) * 255u);
            }
          }
          // Pairs of keys per head dim: {k0 d0, k1 d0, k0 d1, k1 d1}, {.. d2, .. d3} and the same of k2, k3.
          uint32_t va[4], vb[4];
          widen4(__byte_perm(w[0], w[1], 0x5140), va[0], va[1]);
          widen4(__byte_perm(w[2], w[3], 0x5140), va[2], va[3]);
          widen4(__byte_perm(w[0], w[1], 0x7362), vb[0], vb[1]);
          widen4(__byte_perm(w[2], w[3], 0x7362), vb[2], vb[3]);
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            mma_f16(o[2 * dg][n], va, pb[mk][n][0], pb[mk][n][1]);
            mma_f16(o[2 * dg + 1][n], vb, pb[mk][n][0], pb[mk][n][1]);
          }
        }
        // A NaN times a masked probability's zero would reach rows that do not see its token, so such
        // codes went in as zeros; the rows that see them get their NaN here.
        if (!kWhole && __any_sync(0xffffffffu, nans != 0)) {
          for (int kk = 0; kk < 16; ++kk) {
            const int row = 16 * mk + kk;
            if (key + row >= it.s.len) break;
#pragma unroll
            for (int dg = 0; dg < kD / 32; ++dg) {
              const uint32_t bad = nan_bytes(v_word(row, dg));
#pragma unroll
              for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                  for (int q = 0; q < 4; ++q)
                    if (key + row < lim[n][e] && ((bad >> (8 * q + 7)) & 1u))
                      o[2 * dg + (q >> 1)][n][2 * (q & 1) + e] = __uint_as_float(0x7FC00000u);
            }
          }
        }
      }
      release(2 * i + 1);
    };
    int i = 0;
    for (; i < my_tiles && ok; ++i) {
      if (!landed()) break;
      const float4 h0 = meta[2 * (i % C::kMetas)], h1 = meta[2 * (i % C::kMetas) + 1];
      if (fmaxf(fabsf(h0.y), fabsf(h1.y)) > kSameExp) break;
      const int key = key0 + (i * kKW + kw) * kTile;
      if (key + kTile <= full_end && __float_as_uint(h0.w) == 3u)
        tile(std::true_type{}, std::false_type{}, i, key, h0, h1);
      else
        tile(std::false_type{}, std::false_type{}, i, key, h0, h1);
    }
    // From the first tile of far scales on.  (A loop of its own: among the other tiles' code it cost 3 short sequences
    // 6.2 -> 6.4 us, as a call from there as much.)
    if (i < my_tiles && ok) {
      far = true;
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if (g == 0) s_m[kw * kRows + rw * C::kRowsPerWarp + n * 8 + 2 * t + e] = m[n][e];
          m[n][e] = m[n][e] == -INFINITY ? -INFINITY : 0.0f;
        }
      __syncwarp();
      for (; i < my_tiles && ok; ++i) {
        if (!landed()) break;
        const float4 h0 = meta[2 * (i % C::kMetas)], h1 = meta[2 * (i % C::kMetas) + 1];
        tile(std::false_type{}, std::true_type{}, i, key0 + (i * kKW + kw) * kTile, h0, h1);
      }
    }

    // ---------------------------------------------------------------- join the key groups
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 4);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 8);
        l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], 16);
        const int r = rw * C::kRowsPerWarp + n * 8 + 2 * t + e;
        if (g == 0) {
          if (!far) s_m[kw * kRows + r] = m[n][e];
          s_l[kw * kRows + r] = l[n][e];
        }
      }
    // Every tile has been read: the ring's memory is free.  Where a warp gave up a wait the CTA ends, once its copies
    // have landed.
    if (__syncthreads_or(!ok)) {
      if (rw == 0)
        for (int i = 0; i < kSlots; ++i) mbar_wait_warp(&full[i], i < p_slot ? p_phase : p_phase ^ 1);
      return;
    }
    float* merge = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = rw * C::kRowsPerWarp + n * 8 + 2 * t + e;
        float mx = s_m[r];
#pragma unroll
        for (int k = 1; k < kKW; ++k) mx = fmaxf(mx, s_m[k * kRows + r]);
        const float w = mx == -INFINITY ? 1.0f : exp2f(far ? m[n][e] + (s_m[kw * kRows + r] - mx) : m[n][e] - mx);
        float* dst = merge + (size_t)(kw * kRows + r) * C::kPitch + 4 * g;
#pragma unroll
        for (int dg = 0; dg < kD / 32; ++dg)
          *reinterpret_cast<float4*>(dst + dg * 32) = make_float4(o[2 * dg][n][e] * w, o[2 * dg][n][2 + e] * w,
                                                                  o[2 * dg + 1][n][e] * w, o[2 * dg + 1][n][2 + e] * w);
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
        sum += times(s_l[k * kRows + r], pow2_of(mx == -INFINITY ? 0.0f : s_m[k * kRows + r] - mx));
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

template <class C>
cudaError_t launch_cfg(const AttnKv8Launch& L, cudaStream_t stream) {
  auto kern = k_attn_kv8<C>;
  static PerDevice occ = {};
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
  const AttnArgs a = attn_args(L, slots < kMaxRuns ? slots : kMaxRuns);

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
  return launch_join<C>(L, a, stream);
}

// Rows of an item by the most rows a sequence can have (queries times heads per kv head).
template <int kD>
cudaError_t launch_rows(const AttnKv8Launch& L, cudaStream_t stream) {
  const long long rows = (long long)L.max_q_len * (L.q_heads / L.kv_heads);
  // Up to two 8-row tiles per warp (three in the widest form) keep the accumulators, kD / 4 registers
  // each, beside 12 warps per SM; further rows take further warps that read the same tiles.
  constexpr int kSlots = kD == 64 ? 4 : 3;
  if (rows <= 8) return launch_cfg<AttnCfg<kD, 1, 1, 4, kSlots, kD == 256 ? 2 : 4>>(L, stream);
  if (rows <= 16) return launch_cfg<AttnCfg<kD, 2, 1, 4, kSlots, kD == 256 ? 1 : 3>>(L, stream);
  if (rows <= 32 || kD == 256) return launch_cfg<AttnCfg<kD, 2, 2, 2, 4, kD == 256 ? 1 : 3>>(L, stream);
  return launch_cfg<AttnCfg<kD == 256 ? 128 : kD, 3, 2, 2, 4, kD == 64 ? 3 : 2>>(L, stream);
}

int rows_per_item(long long rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 48; }

}  // namespace

size_t attn_kv8_workspace_bytes(int max_q_len, int q_heads, int kv_heads, int head_dim) {
  const size_t rows = (size_t)rows_per_item((long long)max_q_len * (q_heads / kv_heads));
  return 2 * (size_t)kMaxRuns * rows * ((size_t)head_dim + 2) * sizeof(float);
}

cudaError_t launch_attn_kv8(const AttnKv8Launch& L, cudaStream_t stream) {
  switch (L.head_dim) {
    case 64: return launch_rows<64>(L, stream);
    case 128:
      // The other kernel's items cost more beside their keys, so it takes the calls whose page tables allow long
      // sequences (the lengths are not known here).  Measured, this kernel and that: 128 sequences of up to 2000
      // tokens 62 and 70 us, of up to 500 40 and 44 us, 64 of up to 400 with 40 rows 35 and 50 us; 64 of up to
      // 8192 125 and 103 us, 16 of up to 4000 with 320 rows 167 and 96 us.
      if ((long long)L.max_pages * L.page_size > 2048) return launch_attn_kv8_tc(L, stream);
      return launch_rows<128>(L, stream);
    case 256: return launch_rows<256>(L, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace batq
