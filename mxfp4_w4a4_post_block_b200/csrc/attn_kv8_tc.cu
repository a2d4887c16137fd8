// k_attn_kv8_tc: attention over the 8-bit paged cache (attn_kv8.cu has the definition) for head dim 128 and
// long page tables, on block-scaled 8-bit matrix instructions (kind::mxf8f6f4, M = 128).
//
//   S^T = K Q^T     128 keys on the M side, the queries' rows on the N side
//   O^T = V^T P^T   128 head dims on the M side; V's tile as it lies in the cache is the transposed operand
//
// K and V enter as the E4M3 codes that they are, straight from memory by TMA: widening them to f16 in
// registers (attn_kv8.cu) takes most of that kernel's instructions.  What must be more exact than E4M3 is
// written as a sum of E4M3 values whose products add up in one accumulator:
//  - a query as two parts (fp32: three), each 16 times what the ones before leave, four significant bits
//    each, with a scale of its own for every 32 head dims;
//  - a probability as a 20-bit integer's five base-16 digits.  E4M3's codes 0 to 15 are the numbers 0 to 15
//    times 2^-9, so a digit is its own code, and splitting 32 bits into bytes of digits takes two byte
//    permutes and a mask per four values, where conversions run at a quarter of that rate.  The integers
//    count from a power of two above the largest product of probability and V scale among a row's 32 keys,
//    the block's scale takes the difference to the row's reference exponent, and the fp32 accumulators can
//    grow by 2^48 past the reference before it has to move.  A weight is off by 2^-21 of that power of two.
// The page factors: K's multiplies the scores; V's exponent ev is added to them, w = 2^(x + ev), and the sum
// takes w 2^-ev, or where a page's ev is beyond kFarExp exponentials of its own.
//
// An instruction with few columns costs the reading of its 128 x 32 bytes of K or V (45 to 80 clocks), whatever
// its columns: so the parts and digits are columns of their own, all of them up to 24 rows (8 instructions per
// tile instead of 28; 64 sequences of up to 8192 tokens 139 -> 111 us, 16 of up to 16000 with 24 rows 47 -> 39),
// two of them above (16 instructions; 40 rows 68 -> 62 us).
//
// Softmax: a thread has one key of the tile and all rows, so a row's largest of a warp's 32 keys is one
// redux instruction, and its digits of 16 rows are 16 bytes: P is the N-major operand, one store per digit.
//
// A CTA has a load warp (tiles of 128 keys, K and V in turn, a ring of 16 KB slots; page ids read two fetches
// ahead, their factors one), an MMA warp, and one or two groups of four softmax warps that write the outputs
// too.  Up to 16 rows two CTAs share an SM; above, two groups take the tiles in turn with accumulators of
// their own, joined through shared memory (one group took 162 us where two took 118, 16 sequences of up to
// 16000 tokens with 40 rows).  The work list, the runs and the join are attn_kv8.cuh's; an item counts kOver
// units beside its keys (0 -> 4 and 12: 109 -> 100 us and 86 -> 72 us in those cases).
//
// Measured: 64 x up to 8192 tokens, 8 heads of 4 queries: 103 us, 5.7 TB/s; one sequence of 131072: 51 us,
// 5.3 TB/s; both close to the memory's rate.  16 x up to 16000 tokens with 40 rows: 62 us, where the chain of
// a tile bounds it (scores, softmax of 40 rows per key, products; memory 20 us).
#include "attn_kv8.cuh"

namespace batq {
namespace {

constexpr int kTcTile = 128;             // keys per tile
constexpr int kSlotBytes = kTcTile * 128;
constexpr int kQParts = 3;               // of queries (two hold bf16's eight bits)
constexpr int kPParts = 5;               // digits of probabilities
constexpr int kUnits = 3;                // scales of V's rows: 2^-8i
constexpr int kSfAtom = 512;
constexpr int kMeta = 8;                 // tiles whose page factors are kept
constexpr float kWeightUnit = 32.0f;     // weights count 2^-5: 20 bits, and the digits' codes 2^-25
constexpr float kNoRef = -3.0e38f;       // no key seen yet
constexpr float kRise = 48.0f;           // exponent that the accumulators may grow past their reference
constexpr float kMostRise = kRise + 127.0f - kFarExp;  // of a block's scale: V exponents count in full there
constexpr float kLeastRise = -111.0f;    // what lies below has fewer digits (the lowest one's scale is 2^-127)

// kLive: rows of an item; kGroups: groups of four softmax warps, which take the tiles in turn and have
// accumulators each; kSlots: ring slots; kCtas: CTAs per SM.
template <int kLive, int kGroups_, int kSlots_, int kCtas_, int kOver_>
struct TcCfg {
  static constexpr int kOver = kOver_;
  static constexpr float kOutUnit = kWeightUnit;  // what the accumulators and partials count
  static constexpr int kD = 128, kRows = kLive, kUnit = kTcTile, kGroups = kGroups_, kSlots = kSlots_, kCtas = kCtas_;
  // Up to 24 rows, the parts of a row are columns of their own, so that an instruction reads its tile of K or V
  // once for all of them.  Above, TMEM has room for two of them: K's instructions take the first two parts
  // together, and V's two digits at a time, in units 2^8 apart.
  static constexpr bool kStacked = kLive <= 24;
  static constexpr int kRowsN = kStacked ? kLive : (kLive + 15) / 16 * 16;                    // columns of a part
  static constexpr int kNQ = kStacked ? (kQParts * kLive + 15) / 16 * 16 : 2 * kRowsN;        // columns of scores
  static constexpr int kNP = kStacked ? (kPParts * kLive + 15) / 16 * 16 : 2 * kRowsN;        // of accumulators
  static constexpr int kSumParts = kStacked ? kPParts : 2;                                    // that add up
  static constexpr int kWarps = 4 * kGroups;
  static constexpr int kThreads = 32 * (kWarps + 2);
  static constexpr int kQBytes = kStacked ? kNQ * 128 : kQParts * kRowsN * 128;
  static constexpr int kPBytes = kStacked ? kNP * 128 : kPParts * kRowsN * 128;  // a buffer of P
  static constexpr int kQOffset = kSlots * kSlotBytes;
  static constexpr int kPOffset = kQOffset + kQBytes;
  static constexpr int kSfOffset = kPOffset + 2 * kPBytes;     // Q's parts, P's two buffers, the units
  static constexpr int kMetaOffset = kSfOffset + (2 + 2 + kUnits) * kSfAtom;
  static constexpr int kRowOffset = kMetaOffset + kMeta * 8 * 16;
  // Per warp and row: maxima, weights' exponents, sums.  Per group and row: reference, its change.  Per row: keys
  // that it sees, four words of NaN bits, the unit of its scores.
  static constexpr int kBarOffset = kRowOffset + (3 * kWarps + 2 * kGroups + 6) * kLive * 4;
  static constexpr int kBars = 2 * kSlots + 12;
  static constexpr int kSmemBytes = kBarOffset + kBars * 8 + 16 * 4 + 1024;
  static constexpr int kQAtoms = kStacked ? 1 : 2;
  // TMEM columns: scores [2], accumulators [kGroups], scales
  static constexpr int kSStride = (kNQ + 31) / 32 * 32, kOStride = (kNP + 31) / 32 * 32;
  static constexpr int kTO = 2 * kSStride, kTUnit = kTO + kGroups * kOStride, kTQ = kTUnit + 4 * (kStacked ? 1 : kUnits),
                       kTP = kTQ + 4 * kQAtoms;
  static constexpr int kTmem = kTP + 8 <= 256 ? 256 : 512;
  static_assert(kTP + 8 <= 512 && kTmem * kCtas <= 512 && kBarOffset % 8 == 0 && kQBytes % 1024 == 0 && kPBytes % 1024 == 0,
                "layout");
  static_assert(kLive * 128 * 4 <= kPBytes, "a buffer of P holds a group's accumulators");
};

// Maximum over the warp; NaN is passed over.
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ void group_sync(int id) {
  __syncwarp();
  asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}
// Whether any thread of the group says so.
__device__ __forceinline__ bool group_any(int id, bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}
template <int kThreads>
__device__ __forceinline__ void groups_sync() {
  __syncwarp();
  asm volatile("bar.sync 3, %0;" ::"n"(kThreads) : "memory");
}

// Descriptor of one digit of P: 16 rows of a key are 16 bytes, keys follow each other, so it is the N-major
// operand without swizzle: groups of eight keys 128 bytes apart (leading offset), of 16 rows 2048 (stride).
__device__ __forceinline__ uint64_t sdesc_digit(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128u >> 4) << 16) | ((uint64_t)(2048u >> 4) << 32) |
         ((uint64_t)1u << 46);
}

// Base-16 digits of four integers of at most 2^20, digit d of all four in word d.
__device__ __forceinline__ void digits4(const uint32_t (&p)[4], uint32_t (&d)[5]) {
  const uint32_t a = __byte_perm(p[0], p[1], 0x5140), b = __byte_perm(p[2], p[3], 0x5140);
  const uint32_t lo = __byte_perm(a, b, 0x5410), hi = __byte_perm(a, b, 0x7632);
  d[0] = lo & 0x0F0F0F0Fu;
  d[1] = (lo >> 4) & 0x0F0F0F0Fu;
  d[2] = hi & 0x0F0F0F0Fu;
  d[3] = (hi >> 4) & 0x0F0F0F0Fu;
  d[4] = __byte_perm(__byte_perm(p[0], p[1], 0x0062), __byte_perm(p[2], p[3], 0x0062), 0x5410);
}

// Eight consecutive fp32 columns of this thread's TMEM lane, without waiting, and back.
__device__ __forceinline__ void tmem_ld_8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st_8(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}
template <int kCount>
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, float (&v)[kCount]) {
#pragma unroll
  for (int c = 0; c < kCount; c += 8) tmem_ld_8(taddr + c, v + c);
  tmem_ld_wait();
#pragma unroll
  for (int c = 0; c < kCount; ++c) asm volatile("" : "+f"(v[c]));  // not used ahead of the wait
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
    k_attn_kv8_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const AttnArgs a,
                  const int q_bf16) {
  constexpr int kLive = C::kRows, kSlots = C::kSlots, kGroups = C::kGroups, kWarps = C::kWarps;
  constexpr int kAll = 128 * kGroups;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* s_q = smem + C::kQOffset;
  uint8_t* s_p = smem + C::kPOffset;
  uint8_t* s_sfq = smem + C::kSfOffset;
  uint8_t* s_sfp = s_sfq + 2 * kSfAtom;
  uint8_t* s_unit = s_sfp + 2 * kSfAtom;                                 // [kUnits] scales of K's and V's rows
  float4* s_meta = reinterpret_cast<float4*>(smem + C::kMetaOffset);     // [kMeta][8 pages] K scale, V exponent, -, named
  float* s_mx = reinterpret_cast<float*>(smem + C::kRowOffset);          // [kWarps][kLive] exponents of a warp's largest
  float* s_nb = s_mx + kWarps * kLive;                                   // [kWarps][kLive] 20 minus that of the weights
  float* s_l = s_nb + kWarps * kLive;                                    // [kWarps][kLive]
  float* s_fac = s_l;                                                    // [kWarps][kLive] factors of a warp's weights in its sums
  float* s_ref = s_l + kWarps * kLive;                                   // [kGroups][kLive] reference exponents
  float* s_chg = s_ref + kGroups * kLive;                                // [kGroups][kLive] what their change multiplies by, with s_fac
  int* s_lim = reinterpret_cast<int*>(s_chg + kGroups * kLive);          // [kLive] keys that a row sees
  uint32_t* s_nan = reinterpret_cast<uint32_t*>(s_lim + kLive);          // [kLive][4] head dims that are NaN
  float* s_row = reinterpret_cast<float*>(s_nan + 4 * kLive);            // [kLive] units of the rows' scores, where they differ
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
  uint64_t* empty = full + kSlots;
  uint64_t* s_full = empty + kSlots;   // [2] scores are in TMEM
  uint64_t* s_empty = s_full + 2;
  uint64_t* p_full = s_empty + 2;      // [2] probabilities are in shared memory
  uint64_t* p_empty = p_full + 2;
  uint64_t* q_ready = p_empty + 2;
  uint64_t* o_full = q_ready + 1;
  uint64_t* o_empty = o_full + 1;
  uint64_t* all_done = o_empty + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(all_done + 1);
  volatile int* s_bad = reinterpret_cast<volatile int*>(tmem_holder + 1);  // [kGroups] a softmax warp gave up
  int* s_exp = reinterpret_cast<int*>(tmem_holder + 3);                    // [kWarps] exponents of the queries

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    tma_prefetch_map(&tm_k);
    tma_prefetch_map(&tm_v);
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&p_empty[i], 1);
    }
    mbar_init(q_ready, kWarps);
    mbar_init(o_full, 1);
    mbar_init(o_empty, kWarps);
    mbar_init(all_done, 1);
    s_bad[0] = 0;
    s_bad[1] = 0;
    fence_barrier_init();
  }
  // The rows of K have the scale 1, those of V the unit of the digits that they meet.
  if (tid < 128)
    for (int i = 0; i < kUnits; ++i)
      reinterpret_cast<uint32_t*>(s_unit + i * kSfAtom)[tid] = 0x7F7F7F7Fu - (uint32_t)i * 0x08080808u;
  fence_proxy_async_smem();
  if (warp == kWarps + 1) {
    tmem_alloc(tmem_holder, C::kTmem);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;

  // This CTA's run of the work list; every warp walks its items.
  const Runs runs = runs_of(count_units<C>(a, 0, lane).x, a.runs);
  const int u_begin = runs.begin(blockIdx.x), u_end = (int)blockIdx.x < runs.count ? runs.begin(blockIdx.x + 1) : u_begin;
  int b = 0, base_u = 0;
  if (u_begin < u_end) {
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      const int n = b0 + lane < a.batch ? items_of<C>(a, b0 + lane).units(a.kv_heads) : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, n > 0 && base_u + incl > u_begin);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b = b0 + src;
        base_u += __shfl_sync(0xffffffffu, incl - n, src);
        break;
      }
      base_u += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  // A piece of an item: keys [key0, key_end) in `tiles` tiles.
  struct Piece {
    Items it;
    bool first;  // the run's first item
    int b, rt, h, kb0, kb1, rows, lim0, key0, key_end, full_end, tiles;
  };
  // The next piece with keys from unit u on, and u behind it; false behind the run's last.
  auto next_piece = [&](int& u, Piece& p) {
    while (u < u_end) {
      p.it = items_of<C>(a, b);
      while (u - base_u >= p.it.units(a.kv_heads)) {
        base_u += p.it.units(a.kv_heads);
        p.it = items_of<C>(a, ++b);
      }
      const int item = (u - base_u) / p.it.item, from = (u - base_u) - item * p.it.item;
      const int to = min(p.it.item, from + (u_end - u));
      p.b = b;
      p.h = item / p.it.row_tiles;
      p.rt = item - p.h * p.it.row_tiles;
      p.first = u - from <= u_begin;
      u += to - from;
      p.kb0 = max(from - C::kOver, 0);
      p.kb1 = to - C::kOver;
      if (p.kb1 <= p.kb0) continue;
      p.rows = min(kLive, p.it.s.count * a.group - p.rt * kLive);
      p.lim0 = p.it.s.len - p.it.queries + 1;
      p.full_end = p.lim0 + p.rt * kLive / a.group;  // keys that every row sees
      p.key_end = min(min(p.kb1 * kTcTile, p.it.s.len), p.lim0 + (p.rt * kLive + p.rows - 1) / a.group);
      p.key0 = p.kb0 * kTcTile;
      p.tiles = p.key_end > p.key0 ? (p.key_end - p.key0 + kTcTile - 1) / kTcTile : 0;
      return true;
    }
    return false;
  };

  bool ok = true;
  int tile0 = 0;  // tiles before the piece
  if (warp == kWarps) {
    // ------------------------------ loads ------------------------------
    const int np_shift = 7 - a.page_shift, np = 1 << np_shift;  // pages per tile
    const int per_fetch = 32 >> np_shift;                       // tiles that one fetch covers
    int slot = 0, fills = 0;
    uint32_t ph = 0;
    int u = u_begin;
    for (Piece p; ok && next_piece(u, p);) {
      // Lane l: page l % np of tile l / np of a fetch.  Page ids are read two fetches ahead, their scales one.
      auto id_of = [&](int i) {
        const int key = p.key0 + (i + (lane >> np_shift)) * kTcTile + ((lane & (np - 1)) << a.page_shift);
        const int id = key < p.key_end ? a.page_table[(size_t)p.b * a.max_pages + (key >> a.page_shift)] : -1;
        return id < a.num_pages ? id : -1;
      };
      int id = id_of(0), next_id = id_of(per_fetch), ahead_id = -1;
      int ks = 0, vs = 0, next_ks = 0, next_vs = 0;
      if (id >= 0) {
        ks = a.k_scales[id * a.kv_heads + p.h];
        vs = a.v_scales[id * a.kv_heads + p.h];
      }
      for (int i = 0; i < p.tiles && ok; ++i) {
        const int turn = i & (per_fetch - 1);
        if (turn == 0) {
          if (i > 0) {
            id = next_id;
            ks = next_ks;
            vs = next_vs;
            next_id = ahead_id;
          }
          if (next_id >= 0) {
            next_ks = a.k_scales[next_id * a.kv_heads + p.h];
            next_vs = a.v_scales[next_id * a.kv_heads + p.h];
          }
          ahead_id = id_of(i + 2 * per_fetch);
        }
        const int y = id >= 0 ? (id * a.kv_heads + p.h) * a.page_size : -1;
        const float4 f = id >= 0 ? make_float4(vs == 255 ? __uint_as_float(0x7FC00000u) : e8m0_value((uint32_t)ks),
                                               (float)(vs - 127), 0.0f, __int_as_float(1))
                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const bool mine = (lane >> np_shift) == turn;
        const unsigned named = __ballot_sync(0xffffffffu, mine && y >= 0);
        const uint32_t bytes = (uint32_t)__popc(named) * (uint32_t)(a.page_size * 128);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (!mbar_wait_warp(&empty[slot], ph ^ 1)) {
            if (lane == 0) set_error(a.err, kErrReleaseTimeout);
            ok = false;
            break;
          }
          if (kv == 0 && mine) s_meta[((tile0 + i) & (kMeta - 1)) * 8 + (lane & (np - 1))] = f;
          __syncwarp();
          if (lane == 0) mbar_arrive_expect_tx(&full[slot], bytes);
          __syncwarp();
          if (mine && y >= 0)
            tma_load_2d(smem + slot * kSlotBytes + ((lane & (np - 1)) << (a.page_shift + 7)), kv == 0 ? &tm_k : &tm_v,
                        &full[slot], 0, y);
          ++fills;
          if (++slot == kSlots) {
            slot = 0;
            ph ^= 1;
          }
        }
      }
      tile0 += p.tiles;
    }
    // Every copy has landed before the CTA may end, given up or not.
    for (int i = max(0, fills - kSlots); i < fills; ++i)
      if (!mbar_wait_warp(&full[i % kSlots], (i / kSlots) & 1) && lane == 0) set_error(a.err, kErrDataTimeout);
  } else if (warp == kWarps + 1) {
    // ------------------------------ MMA issuer ------------------------------
    // The whole warp runs the loop; one elected lane issues.  The scores of the next kGroups tiles go out
    // before the products with a tile's probabilities.
    const bool issuer = elect_one();
    const int q_parts = q_bf16 ? 2 : kQParts;
    const int n_q = C::kStacked ? (q_parts * kLive + 15) / 16 * 16 : C::kNQ;
    const int q_atoms = C::kStacked ? 1 : q_parts - 1;
    if (issuer)
      for (int i = 0; i < (C::kStacked ? 1 : kUnits); ++i)
        tc_cp_32x128b_warpx4(tmem + C::kTUnit + 4 * i, sdesc_sf_atom(smem_u32(s_unit + i * kSfAtom)));
    __syncwarp();
    int pieces = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok && !mbar_wait_warp(bar, parity)) {
        if (issuer) set_error(a.err, kErrDataTimeout);
        ok = false;
      }
      return ok;
    };
    int u = u_begin;
    for (Piece p; ok && next_piece(u, p);) {
      if (p.tiles == 0) continue;
      if (!wait(q_ready, pieces & 1)) break;
      tc_fence_after_sync();
      if (issuer)
        for (int i = 0; i < q_atoms; ++i)
          tc_cp_32x128b_warpx4(tmem + C::kTQ + 4 * i, sdesc_sf_atom(smem_u32(s_sfq + i * kSfAtom)));
      __syncwarp();
      for (int i = -kGroups; i < p.tiles; ++i) {
        if (i + kGroups < p.tiles) {
          const int g = tile0 + i + kGroups, buf = g & 1, slot = 2 * g % kSlots;
          if (!wait(&full[slot], (2 * g / kSlots) & 1) || !wait(&s_empty[buf], ((g >> 1) & 1) ^ 1)) break;
          tc_fence_after_sync();
          if (issuer) {
            const uint64_t dk = sdesc_kmajor_sw128(smem_u32(smem + slot * kSlotBytes));
            const uint64_t dq = sdesc_kmajor_sw128(smem_u32(s_q));
            const uint32_t t_s = tmem + buf * C::kSStride;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tc_mma_mxf8(t_s, dk + (uint64_t)(j * 2), dq + (uint64_t)(j * 2), idesc_mxf8(128, n_q, 0, j),
                          tmem + C::kTUnit, tmem + C::kTQ, j > 0 ? 1u : 0u);
            if constexpr (!C::kStacked) {
              if (q_parts == 3) {  // the third part joins the first one's columns
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  tc_mma_mxf8(t_s, dk + (uint64_t)(j * 2), dq + (uint64_t)((2 * C::kRowsN * 128 >> 4) + j * 2),
                              idesc_mxf8(128, C::kRowsN, 0, j), tmem + C::kTUnit, tmem + C::kTQ + 4, 1u);
              }
            }
            tc_commit(&empty[slot]);
            tc_commit(&s_full[buf]);
          }
          __syncwarp();
        }
        if (i >= 0) {
          const int g = tile0 + i, buf = g & 1, slot = (2 * g + 1) % kSlots;
          if (!wait(&full[slot], ((2 * g + 1) / kSlots) & 1) || !wait(&p_full[buf], (g >> 1) & 1)) break;
          if (i == 0 && !wait(o_empty, (pieces & 1) ^ 1)) break;
          tc_fence_after_sync();
          if (issuer) {
            tc_cp_32x128b_warpx4(tmem + C::kTP + 4 * buf, sdesc_sf_atom(smem_u32(s_sfp + buf * kSfAtom)));
            // V's tile, 32 keys at a time: keys are its rows of 128 bytes, so it is the M-major operand
            // (bit 15), 8-row groups 1024 bytes apart along K; P's digits are N-major (bit 16).
            const uint64_t dv = sdesc_kmajor_sw128(smem_u32(smem + slot * kSlotBytes));
            const uint64_t dp = sdesc_digit(smem_u32(s_p + buf * C::kPBytes));
            const uint32_t t_acc = tmem + C::kTO + (kGroups == 2 ? buf * C::kOStride : 0);
            constexpr uint32_t kMajors = (1u << 15) | (1u << 16);
            if constexpr (C::kStacked) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tc_mma_mxf8(t_acc, dv + (uint64_t)(j * (32 * 128 >> 4)), dp + (uint64_t)(j * (32 * 16 >> 4)),
                            idesc_mxf8(128, C::kNP, 0, j) | kMajors, tmem + C::kTUnit, tmem + C::kTP + 4 * buf,
                            (i >= kGroups || j > 0) ? 1u : 0u);
            } else {
#pragma unroll
              for (int digit = 0; digit < kPParts; digit += 2)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  tc_mma_mxf8(t_acc, dv + (uint64_t)(j * (32 * 128 >> 4)),
                              dp + (uint64_t)(digit * (C::kRowsN * 128 >> 4) + j * (32 * 16 >> 4)),
                              idesc_mxf8(128, (digit + 1 < kPParts ? 2 : 1) * C::kRowsN, 0, j) | kMajors,
                              tmem + C::kTUnit + 4 * (2 - digit / 2), tmem + C::kTP + 4 * buf,
                              (i >= kGroups || digit > 0 || j > 0) ? 1u : 0u);
            }
            tc_commit(&empty[slot]);
            tc_commit(&p_empty[buf]);
            if (i + 1 == p.tiles) tc_commit(o_full);
          }
          __syncwarp();
        }
      }
      tile0 += p.tiles;
      ++pieces;
    }
    // All instructions have ended before TMEM is freed, given up or not.
    if (issuer) tc_commit(all_done);
    __syncwarp();
    if (!mbar_wait_warp(all_done, 0) && issuer) set_error(a.err, kErrMmaTimeout);
  } else {
    // ------------------------------ softmax and outputs ------------------------------
    const int group = warp >> 2, w4 = warp & 3, gtid = tid & 127, bar_id = 1 + group;
    const uint32_t lanes = (uint32_t)(32 * w4) << 16;  // this warp's TMEM lanes
    float* const ref_of = s_ref + group * kLive;
    float* const chg_of = s_chg + group * kLive;
    float* const mx_of = s_mx + group * 4 * kLive;
    float* const nb_of = s_nb + warp * kLive;
    float* const fac_of = s_fac + warp * kLive;
    float* const also_of = s_fac + group * 4 * kLive;  // (the first warp's factors have no other use meanwhile)
    const uint32_t t_o = tmem + C::kTO + group * C::kOStride + lanes;
    int pieces = 0;
    bool bad = false;  // this warp gave up a wait; its group leaves together (ok)
    auto wait = [&](uint64_t* bar, uint32_t parity, unsigned code) {
      if (!bad && !mbar_wait_warp(bar, parity)) {
        if (lane == 0) set_error(a.err, code);
        bad = true;
      }
    };
    // A piece's queries, four head dims of a row per lane (rows behind its last read that one, so that no load
    // waits): read before the piece ahead of it is written out.
    constexpr int kMine = kLive / kWarps;
    float qv[kMine][4];
    auto load_queries = [&](const Piece& p) {
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const int rr = p.rt * kLive + min(warp + kWarps * k, p.rows - 1);
        const int query = rr / a.group;
        const size_t at =
            (size_t)(p.it.s.begin + query) * (size_t)a.ldq + (size_t)(p.h * a.group + rr - query * a.group) * 128 + lane * 4;
        if (q_bf16) {
          const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.Q) + at);
          qv[k][0] = __uint_as_float(w.x << 16);
          qv[k][1] = __uint_as_float(w.x & 0xFFFF0000u);
          qv[k][2] = __uint_as_float(w.y << 16);
          qv[k][3] = __uint_as_float(w.y & 0xFFFF0000u);
        } else {
          const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(a.Q) + at);
          qv[k][0] = w.x;
          qv[k][1] = w.y;
          qv[k][2] = w.z;
          qv[k][3] = w.w;
        }
      }
    };
    constexpr bool kEarly = kLive <= 16;  // (more rows would spill)
    int u = u_begin;
    Piece next = {};
    bool more = next_piece(u, next);
    if (kEarly && more) load_queries(next);
    while (more && ok) {
      const Piece p = next;
      if (!kEarly) load_queries(p);

      // Queries: row r is query r / G, head h * G + r % G.  A lane has four head dims, eight lanes a block of
      // 32 with the scale 2^e, |q| / 2^e < 256; the parts go to [part][row][128 bytes], swizzled.  The largest e
      // of all rows is left to the scores' factor; where blocks lie further than 2^100 apart, each row has a unit
      // of its own, 2^100 below its largest block where that is above 1, and the factor counts as infinite.
      int qe[kMine], top_e = -126, low_e = 127;
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float m = fabsf(qv[k][i]);
          top = m <= 3.402823466e38f ? fmaxf(top, m) : top;
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        qe[k] = max((int)(__float_as_uint(top) >> 23) - 127 - 7, -126);
        top_e = max(top_e, qe[k]);
        if (top > 0.0f) low_e = min(low_e, qe[k]);
      }
      top_e = __reduce_max_sync(0xffffffffu, top_e);
      low_e = __reduce_min_sync(0xffffffffu, low_e);
      if (lane == 0) s_exp[warp] = top_e * 256 + low_e + 126;
      groups_sync<kAll>();
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        top_e = max(top_e, s_exp[k] >> 8);
        low_e = min(low_e, (s_exp[k] & 255) - 126);
      }
      float scale = fabsf(a.scale_log2) * e8m0_value((uint32_t)(top_e + 127));
      const bool wide = (top_e - low_e > 100 && scale != 0.0f) || scale == INFINITY;
      if (wide) scale = INFINITY;
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const int r = warp + kWarps * k;
        float* v = qv[k];
        int unit = top_e;
        if (wide) {
          unit = __reduce_max_sync(0xffffffffu, qe[k]);
          if (unit > 0) unit -= 100;
        }
        if (wide && lane == 0) s_row[r] = fmaxf(fabsf(a.scale_log2) * e8m0_value((uint32_t)(unit + 127)), 1.4e-45f);
        // (the scores' factor stays positive; what lies 2^119 below the unit has no scale, and counts as zero)
        const float f = qe[k] - unit < -119 ? 0.0f : copysignf(e8m0_value((uint32_t)(127 - qe[k])), a.scale_log2);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = fabsf(v[i]) <= 3.402823466e38f ? v[i] * f : __uint_as_float(0x7FC00000u);
#pragma unroll
        for (int part = 0; part < kQParts; ++part) {
          const uint32_t c = e4m3x4(v[0], v[1], v[2], v[3]);
          const int n = part * C::kRowsN + r;  // row of the operand
          *reinterpret_cast<uint32_t*>(s_q + n * 128 + (((lane >> 2) ^ (n & 7)) << 4) + (lane & 3) * 4) = c;
          if ((lane & 7) == 0) {
            const bool third = !C::kStacked && part == 2;
            const int at = third ? r : n;
            s_sfq[(third ? kSfAtom : 0) + (at & 31) * 16 + (at >> 5) * 4 + (lane >> 3)] =
                (uint8_t)max(qe[k] - unit + 127 - 4 * part, 0);
          }
          const float2 lo = e4m3x2_values(c & 0xFFFFu), hi = e4m3x2_values(c >> 16);
          v[0] = (v[0] - lo.x) * 16.0f;
          v[1] = (v[1] - lo.y) * 16.0f;
          v[2] = (v[2] - hi.x) * 16.0f;
          v[3] = (v[3] - hi.y) * 16.0f;
        }
      }
      for (int r = tid; r < kLive; r += kAll) s_lim[r] = min(p.lim0 + (p.rt * kLive + r) / a.group, p.it.s.len);
      for (int r = tid; r < 4 * kLive; r += kAll) s_nan[r] = 0u;
      for (int r = tid; r < kGroups * kLive; r += kAll) s_ref[r] = kNoRef;
      fence_proxy_async_smem();
      groups_sync<kAll>();
      if (lane == 0 && p.tiles > 0) mbar_arrive(q_ready);

      float l[kLive];  // sums of 2^(score - reference) over this thread's keys
#pragma unroll
      for (int r = 0; r < kLive; ++r) l[r] = 0.0f;
      constexpr int kHeld = (kLive + 31) / 32;  // lane l has rows l and l + 32 of what is the warp's
      for (int i = kGroups == 1 ? 0 : (group ^ tile0) & 1; i < p.tiles; i += kGroups) {
        const int g = tile0 + i, buf = g & 1;
        const uint32_t bph = (g >> 1) & 1;
        wait(&s_full[buf], bph, kErrMmaTimeout);
        tc_fence_after_sync();
        float x[kLive];
        tmem_ld_rows(tmem + buf * C::kSStride + lanes, x);
#pragma unroll
        for (int c = 0; c < kLive; c += 8) {
          float y[8];
          tmem_ld_rows(tmem + buf * C::kSStride + lanes + C::kRowsN + c, y);
          if (C::kStacked && !q_bf16) {
            float z[8];
            tmem_ld_rows(tmem + buf * C::kSStride + lanes + 2 * C::kRowsN + c, z);
#pragma unroll
            for (int r = 0; r < 8; ++r) y[r] += z[r];
          }
#pragma unroll
          for (int r = 0; r < 8; ++r) x[c + r] += y[r];
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[buf]);

        const float4 f = s_meta[(g & (kMeta - 1)) * 8 + (gtid >> a.page_shift)];
        const int key = p.key0 + i * kTcTile + gtid;
        const bool named = __float_as_int(f.w) != 0 && key < p.key_end;
        const bool partly = key >= p.full_end || !named;
        float fs = scale * f.x;
        if (fs == 0.0f) fs = 1.17549435e-38f;  // (a masked score stays -inf)
        if (__any_sync(0xffffffffu, partly)) {
#pragma unroll
          for (int r = 0; r < kLive; ++r)
            if (!named || key >= s_lim[r]) x[r] = -INFINITY;
          if (fs != fs) {  // a NaN scale, which leaves -inf alone
#pragma unroll
            for (int r = 0; r < kLive; ++r)
              if (x[r] != -INFINITY) x[r] = fs;
            fs = 1.0f;
          }
          // V of tokens that no row or not every row sees must not reach a row as NaN times zero: what lies
          // behind the sequence counts as zeros, and NaN codes do, their rows and head dims noted for the end.
          const int vs = (2 * g + 1) % kSlots;
          wait(&full[vs], ((2 * g + 1) / kSlots) & 1, kErrDataTimeout);
          if (partly && !bad) {
            uint8_t* row = smem + vs * kSlotBytes + gtid * 128;
            for (int c = 0; c < 8; ++c) {
              uint4* at = reinterpret_cast<uint4*>(row + ((c ^ (gtid & 7)) << 4));
              if (!named) {
                *at = make_uint4(0u, 0u, 0u, 0u);
                continue;
              }
              const uint4 w = *at;
              uint32_t words[4] = {w.x, w.y, w.z, w.w};
              uint32_t nans = 0;  // of the chunk's 16 codes
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t n = nan_bytes(words[q]) >> 7;
                words[q] &= ~(n * 255u);
                nans |= ((n | n >> 7 | n >> 14 | n >> 21) & 15u) << (4 * q);
              }
              if (nans) {
                *at = make_uint4(words[0], words[1], words[2], words[3]);
                for (int r = 0; r < kLive; ++r)
                  if (key < s_lim[r]) atomicOr(&s_nan[4 * r + (c >> 1)], nans << ((c & 1) * 16));
              }
            }
          }
        }

        // The exponent above each row's largest of the warp's keys, and whether a row has outgrown its reference.
        float held[kHeld], local[kHeld], weights[kHeld];
        auto largest = [&](float exponent, float* to, float (&of)[kHeld]) {
#pragma unroll
          for (int r = 0; r < kLive; r += 4) {
            float4 m;
            m.x = redux_max(fmaf(x[r], fs, exponent));
            m.y = redux_max(fmaf(x[r + 1], fs, exponent));
            m.z = redux_max(fmaf(x[r + 2], fs, exponent));
            m.w = redux_max(fmaf(x[r + 3], fs, exponent));
            if (lane == 0) *reinterpret_cast<float4*>(to + r) = m;
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < kHeld; ++k) {
            of[k] = kNoRef;
            if (lane + 32 * k < kLive) of[k] = ceilf(to[lane + 32 * k]);
          }
          __syncwarp();
        };
        // The exponents are taken of rounded scores, the weights' differences of exact ones: so scores that may pass
        // 2^21 (|x| < 2^24) are rounded first, and counted from each row's largest, `base`.
        float base[kHeld];
#pragma unroll
        for (int k = 0; k < kHeld; ++k) base[k] = 0.0f;
        if (__any_sync(0xffffffffu, fs > 0.125f)) {
          // (factors one after the other: their product may leave fp32's range where the score does not)
          const float by = s_meta[(g & (kMeta - 1)) * 8 + (gtid >> a.page_shift)].x;  // f.x again (registers)
          const float before = by > 0.0f && by < 1.0f ? by : 1.0f, after = fs != fs ? fs : fmaxf(by, 1.0f);
#pragma unroll
          for (int r = 0; r < kLive; ++r) x[r] = x[r] * before * (scale == INFINITY ? s_row[r] : scale) * after;
          fs = 1.0f;
          largest(0.0f, nb_of, base);
#pragma unroll
          for (int k = 0; k < kHeld; ++k) {
            base[k] = base[k] > kNoRef ? base[k] : 0.0f;
            if (lane + 32 * k < kLive) nb_of[lane + 32 * k] = base[k];
          }
          __syncwarp();
#pragma unroll
          for (int r = 0; r < kLive; ++r) x[r] -= nb_of[r];
          __syncwarp();
        }
        largest(near_exponent(f.y), mx_of + w4 * kLive, held);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
          weights[k] = local[k] = held[k];
          held[k] += base[k];
        }
        const bool far = __any_sync(0xffffffffu, named && fabsf(f.y) > kFarExp);
        if (far) largest(f.y, nb_of, weights);
        bool outgrown = bad;
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
          const int r = lane + 32 * k;
          if (r < kLive) {
            mx_of[w4 * kLive + r] = held[k];
            nb_of[r] = weights[k] > kNoRef ? 20.0f - weights[k] : 0.0f;
            outgrown |= held[k] > ref_of[r] + kRise;
          }
        }
        if (bad && lane == 0) s_bad[group] = 1;
        if (group_any(bar_id, outgrown)) {
          ok = s_bad[group] == 0;
          float next[kHeld];
#pragma unroll
          for (int k = 0; k < kHeld; ++k) {
            const int r = lane + 32 * k;
            next[k] = kNoRef;
            if (r < kLive) {
              const float top =
                  fmaxf(fmaxf(mx_of[r], mx_of[kLive + r]), fmaxf(mx_of[2 * kLive + r], mx_of[3 * kLive + r]));
              const float ref = ref_of[r];
              next[k] = top > ref + kRise ? top : ref;
              if (w4 == 0) {
                const Pow2 change = pow2_of(ref == kNoRef ? 0.0f : ref - next[k]);
                chg_of[r] = change.a;
                also_of[r] = change.b;
              }
            }
          }
          group_sync(bar_id);
          if (!ok) break;
          if (w4 == 0)
#pragma unroll
            for (int k = 0; k < kHeld; ++k)
              if (lane + 32 * k < kLive) ref_of[lane + 32 * k] = next[k];
          if (i >= kGroups) {
            const int before = g - kGroups;  // the group's last tile: all products so far
            wait(&p_empty[before & 1], (before >> 1) & 1, kErrMmaTimeout);
            tc_fence_after_sync();
            for (int part = 0; part < C::kSumParts; ++part)
              for (int c = 0; c < kLive; c += 8) {
                float o[8];
                tmem_ld_rows(t_o + part * C::kRowsN + c, o);
#pragma unroll
                for (int r = 0; r < 8; ++r) o[r] = o[r] * chg_of[c + r] * also_of[c + r];
                tmem_st_8(t_o + part * C::kRowsN + c, o);
              }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before_sync();
#pragma unroll
            for (int r = 0; r < kLive; ++r) l[r] = l[r] * chg_of[r] * also_of[r];
          }
          group_sync(bar_id);
        }

        // Weights: 2^(x + ev - block + 20), rounded to an integer by the 2^23 added to it (NaN's bits have the
        // top digit 255, a NaN), and its digits, which are E4M3 codes as they stand.
        wait(&p_empty[buf], bph ^ 1, kErrMmaTimeout);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
          const int r = lane + 32 * k;
          if (r < kLive) {
            // (`local` stands at held - reference; all else of the tile goes by its distance from it, since fp32 holds
            // large scores in steps that V's exponents are lost in)
            const float at = local[k] > kNoRef ? held[k] - ref_of[r] : 0.0f;
            float rise = weights[k] > kNoRef ? fminf(at + (weights[k] - local[k]), kMostRise) : 0.0f;
            if (rise < kLeastRise) {
              nb_of[r] += rise - kLeastRise;
              rise = kLeastRise;
            }
            mx_of[w4 * kLive + r] = local[k] > kNoRef ? at - local[k] : 0.0f;
            fac_of[r] = ex2(rise - 20.0f);
            uint8_t* sf = s_sfp + buf * kSfAtom + w4;
            if constexpr (C::kStacked) {
#pragma unroll
              for (int digit = 0; digit < kPParts; ++digit) {
                const int n = digit * kLive + r;
                sf[(n & 31) * 16 + (n >> 5) * 4] = (uint8_t)((int)rise + 127 - 4 * (kPParts - 1 - digit));
              }
            } else {
#pragma unroll
              for (int odd = 0; odd < 2; ++odd) {
                const int n = odd * C::kRowsN + r;
                sf[(n & 31) * 16 + (n >> 5) * 4] = (uint8_t)((int)rise + 127 + 4 * odd);
              }
            }
          }
        }
        __syncwarp();
        // A weight is 2^(20 - rise + ev) times what the sum takes.  V exponents far apart would leave some weights
        // below fp32's range: those sums are taken on their own.
        float unscale = __int_as_float((127 - (int)near_exponent(f.y)) << 23);
        if (far) {
          unscale = 0.0f;
#pragma unroll
          for (int r = 0; r < kLive; ++r) l[r] += ex2(fmaf(x[r], fs, mx_of[w4 * kLive + r]));
        }
        uint8_t* dst = s_p + buf * C::kPBytes + gtid * 16;
#pragma unroll
        for (int r0 = 0; r0 < kLive; r0 += 16) {
          uint32_t d[4][5];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = r0 + 4 * q;
            if (r >= kLive) break;
            const float4 nb = *reinterpret_cast<const float4*>(nb_of + r);
            const float4 fac = *reinterpret_cast<const float4*>(fac_of + r);
            const float v0 = ex2(fmaf(x[r], fs, f.y + nb.x)), v1 = ex2(fmaf(x[r + 1], fs, f.y + nb.y)),
                        v2 = ex2(fmaf(x[r + 2], fs, f.y + nb.z)), v3 = ex2(fmaf(x[r + 3], fs, f.y + nb.w));
            l[r] = fmaf(v0 * unscale, fac.x, l[r]);
            l[r + 1] = fmaf(v1 * unscale, fac.y, l[r + 1]);
            l[r + 2] = fmaf(v2 * unscale, fac.z, l[r + 2]);
            l[r + 3] = fmaf(v3 * unscale, fac.w, l[r + 3]);
            const uint32_t w[4] = {__float_as_uint(v0 + 8388608.0f), __float_as_uint(v1 + 8388608.0f),
                                   __float_as_uint(v2 + 8388608.0f), __float_as_uint(v3 + 8388608.0f)};
            digits4(w, d[q]);
          }
          // Row n of the operand: byte n % 16 of the key's 16 bytes in group n / 16.
          if constexpr (kLive == 8) {  // two digits of eight rows side by side
#pragma unroll
            for (int digit = 0; digit < kPParts; digit += 2) {
              const int second = digit + 1 < kPParts ? digit + 1 : digit;  // (the last one's columns are not read)
              *reinterpret_cast<uint4*>(dst + digit * 1024) =
                  make_uint4(d[0][digit], d[1][digit], d[0][second], d[1][second]);
            }
          } else {
#pragma unroll
            for (int digit = 0; digit < kPParts; ++digit) {
              const int n = digit * C::kRowsN + r0;
              if (n % 16 == 0 && r0 + 16 <= kLive) {
                *reinterpret_cast<uint4*>(dst + n * 128) = make_uint4(d[0][digit], d[1][digit], d[2][digit], d[3][digit]);
              } else {
                *reinterpret_cast<uint2*>(dst + n / 16 * 2048 + n % 16) = make_uint2(d[0][digit], d[1][digit]);
                if (r0 + 16 <= kLive)
                  *reinterpret_cast<uint2*>(dst + (n + 8) / 16 * 2048 + (n + 8) % 16) = make_uint2(d[2][digit], d[3][digit]);
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }

      // ------------------------------ the piece's sums and outputs ------------------------------
#pragma unroll
      for (int r = 0; r < kLive; ++r) {
        float v = l[r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) s_l[warp * kLive + r] = v;
      }
      if (kEarly) {
        more = next_piece(u, next);
        if (more) load_queries(next);
      }
      float* const merge = reinterpret_cast<float*>(s_p + group * C::kPBytes);  // [kLive][128], once P has been read
      const bool any_tile = p.tiles > (kGroups == 1 ? 0 : (group ^ tile0) & 1);
      if (p.tiles > 0 && ok) {
        wait(o_full, pieces & 1, kErrMmaTimeout);
        tc_fence_after_sync();
      }
#pragma unroll
      for (int c = 0; c < kLive; c += 8) {
        float o[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (any_tile && ok) {
          tmem_ld_rows(t_o + c, o);
#pragma unroll
          for (int part = 1; part < C::kSumParts; ++part) {
            float more[8];
            tmem_ld_rows(t_o + part * C::kRowsN + c, more);
#pragma unroll
            for (int r = 0; r < 8; ++r) o[r] += more[r];
          }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) merge[(c + r) * 128 + gtid] = o[r];
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0 && p.tiles > 0 && ok) mbar_arrive(o_empty);
      if (bad && lane == 0) s_bad[group] = 1;
      groups_sync<kAll>();
      ok = s_bad[0] == 0 && s_bad[1] == 0;
      const bool complete = p.kb0 == 0 && p.kb1 == p.it.key_blocks;
      const int part_slot = 2 * blockIdx.x + (p.first ? 0 : 1);
      for (int r = warp; r < p.rows; r += kWarps) {  // a warp per row, four head dims per lane
        float top = s_ref[r], sum = 0.0f;
        if constexpr (kGroups == 2) top = fmaxf(top, s_ref[kLive + r]);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          const float ref = s_ref[k * kLive + r];
          const Pow2 w = pow2_of(ref == kNoRef ? 0.0f : ref - top);  // (a group that saw no key adds its zeros, or NaN)
          const float* lk = s_l + k * 4 * kLive + r;
          sum = fmaf(w.a * (lk[0] + lk[kLive] + lk[2 * kLive] + lk[3 * kLive]), w.b, sum);
          const float4 o = *reinterpret_cast<const float4*>(s_p + k * C::kPBytes + r * 512 + lane * 16);
          v.x = fmaf(w.a * o.x, w.b, v.x);
          v.y = fmaf(w.a * o.y, w.b, v.y);
          v.z = fmaf(w.a * o.z, w.b, v.z);
          v.w = fmaf(w.a * o.w, w.b, v.w);
        }
        const uint32_t nans = s_nan[4 * r + (lane >> 3)] >> ((lane & 7) * 4);
        if (nans & 1u) v.x = __uint_as_float(0x7FC00000u);
        if (nans & 2u) v.y = __uint_as_float(0x7FC00000u);
        if (nans & 4u) v.z = __uint_as_float(0x7FC00000u);
        if (nans & 8u) v.w = __uint_as_float(0x7FC00000u);
        const float m = top == kNoRef ? -INFINITY : top;
        if (complete) {
          const int rr = p.rt * kLive + r, query = rr / a.group;
          const size_t row = (size_t)(p.it.s.begin + query);
          const int head = p.h * a.group + rr - query * a.group;
          const size_t at = row * (size_t)a.ldo + (size_t)head * 128 + lane * 4;
          const float inv = sum == 0.0f ? 0.0f : kWeightUnit / sum;  // a row that sees nothing: zeros
          if (a.out_bf16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
          else
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) =
                make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
          if (a.lse && lane == 0) a.lse[row * a.q_heads + head] = sum == 0.0f ? -INFINITY : kLn2 * (m + log2f(sum));
        } else {
          *reinterpret_cast<float4*>(a.partial + ((size_t)part_slot * kLive + r) * 128 + lane * 4) = v;
          if (lane == 0) {
            float* ml = a.partial + (size_t)2 * a.runs * kLive * 128;
            ml[(size_t)part_slot * kLive + r] = m;
            ml[(size_t)(2 * a.runs + part_slot) * kLive + r] = sum;
          }
        }
      }
      groups_sync<kAll>();  // the next piece writes the row arrays
      tile0 += p.tiles;
      pieces += p.tiles > 0 ? 1 : 0;
      if (!kEarly) more = next_piece(u, next);
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (warp == kWarps + 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::kTmem);
  }
}

template <class C>
cudaError_t launch_tc(const AttnKv8Launch& L, cudaStream_t stream) {
  auto kern = k_attn_kv8_tc<C>;
  static PerDevice attr_set = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_set[dev] = 1;
  }
  const int slots = sm_count() * C::kCtas;
  const AttnArgs a = attn_args(L, slots < kMaxRuns ? slots : kMaxRuns);
  CUtensorMap tm_k, tm_v;
  const uint64_t rows = (uint64_t)L.num_pages * L.kv_heads * L.page_size;
  if (!make_map_2d(&tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.k_codes, 128, rows, 128, 128, L.page_size,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_2d(&tm_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.v_codes, 128, rows, 128, 128, L.page_size,
                   CU_TENSOR_MAP_SWIZZLE_128B))
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tm_k, tm_v, a, L.q_bf16 ? 1 : 0);
  if (e != cudaSuccess) return e;
  return launch_join<C>(L, a, stream);
}

}  // namespace

cudaError_t launch_attn_kv8_tc(const AttnKv8Launch& L, cudaStream_t stream) {
  const long long rows = (long long)L.max_q_len * (L.q_heads / L.kv_heads);
  // Rows in steps of 8, since the softmax's time goes with them (40 rows in an item of 48: 71 us for 16 sequences
  // of up to 16000 tokens instead of 62).  More than 48 go in equal row tiles.  Up to 16 rows two CTAs of 107 KB
  // share an SM; above, it has one with two groups.
  const long long tiles = (rows + 47) / 48, per_tile = (rows + tiles - 1) / tiles;
  if (per_tile <= 8) return launch_tc<TcCfg<8, 1, 5, 2, 4>>(L, stream);
  if (per_tile <= 16) return launch_tc<TcCfg<16, 1, 4, 2, 4>>(L, stream);
  if (per_tile <= 24) return launch_tc<TcCfg<24, 2, 8, 1, 12>>(L, stream);
  if (per_tile <= 32) return launch_tc<TcCfg<32, 2, 8, 1, 12>>(L, stream);
  if (per_tile <= 40) return launch_tc<TcCfg<40, 2, 8, 1, 12>>(L, stream);
  return launch_tc<TcCfg<48, 2, 8, 1, 12>>(L, stream);
}

}  // namespace batq
