// k_linear_w4a16: out = (X P) W'^T for 1 to 16 tokens, 4-bit prepared weights, activations not
// quantised to the weights' width.
//
//   out[s][m] = sum_n w[m][n] y[s][n],    y_s = x_s P  (or x_s itself)
//
// with w the E2M1 codes times their group scales (E8M0 per 32, or E4M3 per 16 and 1 / gs on the
// result: NVFP4).  With so few tokens the weights' bytes are the work, so nothing is done to them:
// they go from memory by TMA straight into block-scaled 4-bit matrix instructions (kind::mxf4,
// kind::mxf4nvf4), 128 weight rows on the M side.  The tokens' precision comes from several columns
// instead of wider elements: y / 2^e, 2^e the scale of y's block, is rounded to a fixed-point number
// and written in radix 8 with the digits -4 .. 3, which are E2M1 values,
//   y = 2^e (d_0 + d_1 / 8 + d_2 / 64 + ..),   |y| < 2 * 2^e,
// one column of the N side per token and digit, all digits of a block under the block's scale, and
// the digits' accumulators are added with the weights 1, 1/8, 1/64, .. in the epilogue.  Six digits
// (2^-16 of the block's largest value, so that a value 2^7 below it still has bf16's bits) serve a bf16
// output, eight (2^-22) an fp32 one; sixteen tokens then are 96 or 128 of the 256 columns an instruction
// can have, and the tensor pipe still waits for memory.  (Five digits are as fast up to four tokens and 2
// to 4 % faster for sixteen, 11.0 instead of 11.5 us for 16 x 4096 x 4096, but lose bits of bf16 tokens
// beside values 2^4 larger, as outlier channels are.  With the weights widened to f16 in registers for m16n8k16 instructions, the same products
// were bound by the conversions: 4 tokens x 4096 x 24576 took 30 us, 16 tokens 113 us.)
//
// A CTA makes its tokens' digits once, keeps them and their scales (shared memory, TMEM), and walks
// 128-row tiles of the weights.  One warp loads stages of K = 256 (16 KB of codes by TMA with the
// 128-byte swizzle, 512-byte scale tiles) into a ring, one copies their scales into TMEM and issues four
// MMAs per stage into one of two accumulators, four drain the other.  Sixteen warps make the digits,
// stage after stage, so the first tile's products begin with the first stage's.  The CTAs of a cluster
// split K where the digits would not fit otherwise or where it balances the tiles over the SMs
// (launch_cfg); each sends its sums straight to the CTA that adds their rows, rank after rank (one way
// through distributed shared memory; fetching them after a barrier of the cluster took 1 to 2 us more).
//
// What bounds it: at one tile per CTA the chain of launch, digits (1.4 us per unit of a warp), products
// and exchange; with many the stream of weights.  Measured: one token x 4096 x 4096 5.7 us (1.5 TB/s; an
// empty kernel's launch takes 2.5), four x 4096 x 24576 13.0 us (4.1 TB/s), seven x 12288 x 4096 NVFP4
// with fp32 out 12.5 us (2.3 TB/s), 16 x 4096 x 24576 23.7 us.
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "host_util.h"
#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace batq {
namespace {

constexpr int kMakerWarps = 16;                  // make the digits; then the first four drain the accumulators
constexpr int kMakers = 32 * kMakerWarps;
constexpr int kLoadWarp = kMakerWarps, kMmaWarp = kMakerWarps + 1;
constexpr int kThreads = 32 * (kMakerWarps + 2);
constexpr int kRows = 128;                       // weight rows per tile
constexpr int kStageK = 256;                     // K elements per stage
constexpr int kStageBytes = kRows * kStageK / 2;
constexpr int kSfAtom = 512;
constexpr int kMaxRing = 10;
constexpr int kMaxPasses = 32;                   // of the makers over their items (the digits' space allows 14)
constexpr int kPartsBf16 = 6, kPartsF32 = 8;     // digits by output type

struct W4Args {
  const void* X;
  int x_bf16, S, N, ldx;
  int transform;
  float A[64], a_norm;        // a_norm: four times the largest column sum of |A|
  const float* B;
  const uint8_t* scales;
  const float* gs;
  int M, groups;              // groups: scale tiles (four scale columns) per 128 rows
  int out_bf16;
  void* out;
  int ldo;
  unsigned* err;
  int tiles, stages, ring;    // 128-row tiles; K stages of a row; ring slots
  int parts, n;               // digits; columns (parts * padded tokens, rounded up to 16)
  int acc_stride, t_sx, t_sw; // TMEM columns: second accumulator, digit scales, weight scales
  int max_stages;             // most stages of a CTA
};

// Eight consecutive elements of token s.
__device__ __forceinline__ void load_x8(const W4Args& a, int s, int k, float (&v)[8]) {
  if (a.x_bf16) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.X) + (size_t)s * a.ldx + k));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.X) + (size_t)s * a.ldx + k);
    const float4 x = __ldg(p), y = __ldg(p + 1);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
  }
}

// Smallest e >= -126 with a < 2 * 2^e, a finite and >= 0.
__device__ __forceinline__ int digit_exponent(float a) { return max((int)(__float_as_uint(a) >> 23) - 127, -126); }

// E2M1 codes of the digit whose three bits (the digit plus four) stand at bit kAt of eight fixed-point
// numbers, v[j] holding number 2 j in its low half and 2 j + 1 in its high half.  The bits select the
// code by byte permutes: even numbers' codes from one table, odd numbers' from the same in the high nibble.
template <int kAt>
__device__ __forceinline__ uint32_t digit_codes(const uint32_t (&v)[4]) {
  uint32_t sel = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t t = kAt >= 4 * j ? v[j] >> (kAt >= 4 * j ? kAt - 4 * j : 0) : v[j] << (kAt < 4 * j ? 4 * j - kAt : 0);
    sel |= t & (0x00070007u << (4 * j));
  }
  constexpr uint32_t kNeg = 0x0A0C0D0Eu, kPos = 0x05040200u;  // codes of -4 .. -1 and of 0 .. 3
  return __byte_perm(kNeg, kPos, sel) | __byte_perm(kNeg << 4, kPos << 4, sel >> 16);
}

// Writes kN floats to a peer's shared memory and counts their bytes on its barrier.
template <int kN>
__device__ __forceinline__ void push_cluster(uint32_t addr, const float* v, uint32_t bar) {
  if constexpr (kN == 1)
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
                 "r"(__float_as_uint(v[0])), "r"(bar)
                 : "memory");
  else if constexpr (kN == 2)
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(addr),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(bar)
                 : "memory");
  else
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(bar)
                 : "memory");
}

// mbar_wait_warp with an acquire at cluster scope.
__device__ __forceinline__ bool mbar_wait_warp_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t done = 0;
  const uint64_t t0 = global_timer_ns();
  do {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendHintNs)
        : "memory");
  } while (!done && global_timer_ns() - t0 <= kWaitLimitNs);
  return __all_sync(0xffffffffu, done != 0) != 0;
}

// Joins the four epilogue warps; whether all of their threads say so.
__device__ __forceinline__ bool all_epilogue(bool v) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// f(0), f(1), .. as compile-time numbers.
template <int kCount, class F, int... kI>
__device__ __forceinline__ void for_digits_impl(F&& f, std::integer_sequence<int, kI...>) {
  (f(std::integral_constant<int, kI>{}), ...);
}
template <int kCount, class F>
__device__ __forceinline__ void for_digits(F&& f) {
  for_digits_impl<kCount>(f, std::make_integer_sequence<int, kCount>{});
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// kN consecutive fp32 columns of this thread's TMEM lane.
template <int kN>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[kN]) {
  static_assert(kN == 1 || kN == 2 || kN == 4 || kN == 8, "columns");
  if constexpr (kN == 1)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r[0]) : "r"(taddr));
  else if constexpr (kN == 2)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
  else if constexpr (kN == 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
  else
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// kSp: tokens padded to a power of two (columns of a digit); kParts: digits.
template <int kSp, bool kNv, int kParts>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_w4a16(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ W4Args a) {
  constexpr int kAtoms = kNv ? 4 : 2;             // scale tiles (four scale columns) of a stage
  constexpr int kSfBytes = kAtoms * kSfAtom;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* s_w = smem;                                                     // [ring] weight codes
  uint8_t* s_x = s_w + a.ring * kStageBytes;                               // [stage][column] digits
  uint8_t* s_sw = s_x + (size_t)a.max_stages * a.n * 128;                  // [ring] weight scale tiles
  uint8_t* s_sx = s_sw + a.ring * kSfBytes;                                // digit scale tiles
  float* s_sums = reinterpret_cast<float*>(s_sx + a.max_stages * kSfBytes);  // [2][rank][row][kSp]
  float* s_xf = s_sums + 2 * (kRows + 8) * kSp;                                  // [16] NVFP4: each token's unit
  unsigned* s_amax = reinterpret_cast<unsigned*>(s_xf + 16);               // [16]
  uint64_t* full = reinterpret_cast<uint64_t*>(s_amax + 16);
  uint64_t* empty = full + kMaxRing;
  uint64_t* acc_full = empty + kMaxRing;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* sums_ready = acc_empty + 2;
  uint64_t* all_done = sums_ready + 2;                                     // products have ended
  uint64_t* made = all_done + 1;                                           // [kMaxPasses] digits of a pass
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(made + kMaxPasses);

  uint32_t csize, crank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(csize));
  asm("mov.u32 %0, %%cluster_ctaid.x;" : "=r"(crank));
  const int cluster = blockIdx.x / csize, clusters = gridDim.x / csize;
  const int st0 = (int)((long long)a.stages * crank / csize);       // this CTA's K stages
  const int st1 = (int)((long long)a.stages * (crank + 1) / csize);
  const int k0 = st0 * kStageK, k1 = min(st1 * kStageK, a.N);

  if (tid == 0) {
    tma_prefetch_map(&tm_w);
    for (int i = 0; i < a.ring; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(all_done, 1);
    for (int i = 0; i < kMaxPasses; ++i) mbar_init(&made[i], kMakerWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
      mbar_init(&sums_ready[i], 1);
    }
    fence_barrier_init();
  }
  if (tid < 16) s_amax[tid] = 0u;
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  if (csize > 1) cluster_sync_all();  // the peers' barriers are initialised
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;

  if (warp == kLoadWarp) {
    // ------------------------------ loads ------------------------------
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = cluster; tile < a.tiles && ok; tile += clusters)
        for (int st = st0; st < st1; ++st) {
          if (!mbar_wait(&empty[s], ph ^ 1)) {
            set_error(a.err, kErrReleaseTimeout);
            ok = false;
            break;
          }
          const int atoms = min(kAtoms, a.groups - st * kAtoms);
          mbar_arrive_expect_tx(&full[s], (uint32_t)(kStageBytes + atoms * kSfAtom));
          tma_load_2d(s_w + s * kStageBytes, &tm_w, &full[s], st * (kStageK / 2), tile * kRows);
          bulk_load(s_sw + s * kSfBytes, a.scales + ((size_t)tile * a.groups + (size_t)st * kAtoms) * kSfAtom,
                    (uint32_t)(atoms * kSfAtom), &full[s]);
          if (++s == a.ring) {
            s = 0;
            ph ^= 1;
          }
        }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------ scale copies and MMAs ------------------------------
    // One thread's copies and MMAs run in order.  (Another warp issuing the copies a stage ahead, as in
    // the GEMMs with wide tiles, costs a commit and a barrier per stage: 9.8 instead of 8.4 us for one
    // tile of K = 4096; the same thread issuing them ahead of the last stage's MMAs 20 instead of 15 us for
    // four tokens x 4096 x 24576.)  It is that thread's own instructions that take the time, so the loop is
    // its alone, without votes, and has straight-line code for whole stages.
    const bool issuer = elect_one();
    if (issuer) {
    const int whole_stages = a.N / kStageK;
    // What the loop would work out for every stage: it is the issuing thread's own instructions that limit it.
    const uint64_t dw0 = sdesc_kmajor_sw128(smem_u32(s_w)), dx0 = sdesc_kmajor_sw128(smem_u32(s_x));
    const uint64_t dsw0 = sdesc_sf_atom(smem_u32(s_sw)), dsx0 = sdesc_sf_atom(smem_u32(s_sx));
    const uint32_t t_sw0 = tmem + a.t_sw, t_sx0 = tmem + a.t_sx;
    const uint32_t idesc = kNv ? idesc_nvf4(kRows, a.n) : idesc_mxf4(a.n, 0, 0);
    [[maybe_unused]] const uint32_t idesc_odd = idesc_mxf4(a.n, 2, 2);
    int s = 0, it = 0, passes = 0;   // passes: digits known to be made
    uint32_t ph = 0;
    bool ok = true;
    for (int tile = cluster; tile < a.tiles && ok; tile += clusters, ++it) {
      const int buf = it & 1;
      if (!mbar_wait(&acc_empty[buf], ((it >> 1) & 1) ^ 1)) {
        set_error(a.err, kErrDrainTimeout);
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t t_acc = tmem + buf * a.acc_stride;
      for (int st = st0; st < st1; ++st) {
        if (it == 0) {  // the stage's digits and their scales
          const int need = ((st - st0 + 1) * a.S + kMakerWarps - 1) / kMakerWarps;
          for (; passes < need && ok; ++passes) ok = mbar_wait(&made[passes], 0);
        }
        if (!ok || !mbar_wait(&full[s], ph)) {
          set_error(a.err, kErrDataTimeout);
          ok = false;
          break;
        }
        tc_fence_after_sync();
        {
          const uint32_t tsw = t_sw0 + s * (4 * kAtoms), tsx = t_sx0 + (st - st0) * (4 * kAtoms);
          const uint64_t dsw = dsw0 + (uint64_t)(uint32_t)(s * (kSfBytes >> 4));
          const uint64_t dsx = dsx0 + (uint64_t)(uint32_t)((st - st0) * (kSfBytes >> 4));
          const uint64_t dw = dw0 + (uint64_t)(uint32_t)(s * (kStageBytes >> 4));
          const uint64_t dx = dx0 + (uint64_t)(uint32_t)((st - st0) * (a.n * 8));
          auto copy = [&](int i) { tc_cp_32x128b_warpx4(tsw + 4 * i, dsw + (uint64_t)(i * (kSfAtom >> 4))); };
          auto copy_x = [&](int i) { tc_cp_32x128b_warpx4(tsx + 4 * i, dsx + (uint64_t)(i * (kSfAtom >> 4))); };
          auto mma = [&](int j, uint32_t acc) {
            if constexpr (kNv)
              tc_mma_nvf4(t_acc, dw + (uint64_t)(j * 2), dx + (uint64_t)(j * 2), idesc, tsw + 4 * j, tsx + 4 * j, acc);
            else
              tc_mma_mxf4(t_acc, dw + (uint64_t)(j * 2), dx + (uint64_t)(j * 2), (j & 1) ? idesc_odd : idesc,
                          tsw + 4 * (j >> 1), tsx + 4 * (j >> 1), acc);
          };
          const uint32_t later = st > st0 ? 1u : 0u;
          if (st < whole_stages) {
            if (it == 0) {
#pragma unroll
              for (int i = 0; i < kAtoms; ++i) copy_x(i);
            }
#pragma unroll
            for (int i = 0; i < kAtoms; ++i) copy(i);
            mma(0, later);
#pragma unroll
            for (int j = 1; j < 4; ++j) mma(j, 1u);
          } else {
            const int nmma = (a.N - st * kStageK) >> 6, atoms = kNv ? nmma : (nmma + 1) >> 1;
            for (int i = 0; i < atoms; ++i) {
              copy(i);
              if (it == 0) copy_x(i);
            }
            for (int j = 0; j < nmma; ++j) mma(j, j > 0 ? 1u : later);
          }
          tc_commit(&empty[s]);
          if (st == st1 - 1) tc_commit(&acc_full[buf]);
        }
        if (++s == a.ring) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    // All instructions have ended before TMEM is freed, given up or not.
    tc_commit(all_done);
    if (!mbar_wait(all_done, 0)) set_error(a.err, kErrMmaTimeout);
    // Where any role gave up this one does too, and copies may be on their way: each slot's barrier gets its time, in
    // the phase that it is in.  (Waiting for all slots always took 0.5 us of 3.4 for one token x 512 x 512.)
    for (int i = 0; !ok && i < 2 * a.ring; ++i) mbar_wait(&full[i >> 1], i & 1);
    }
  } else {
    // ------------------------------ digits ------------------------------
    // A thread makes row b (eight values) of one 4 x 8 block of one token: u = column b of B^T against
    // the block's four rows, y = u A (A from the parameter bank).  A warp makes 32 rows (8 blocks, a stage)
    // of one token at a time: unit q of the units in the order of the stages, within a stage token after
    // token.  The instructions of that bound the start of a call (a unit of eight digits took 600, and 16
    // warps share four schedulers), so all that is the warp's or the digit's is worked out once for it.
    const int units = (st1 - st0) * a.S;
    const uint32_t per_token = (65536u + (uint32_t)a.S - 1) / (uint32_t)a.S;  // q / S = q * this >> 16 (q < 4096)
    auto stage_of = [&](int q) { return (int)(((uint32_t)q * per_token) >> 16); };
    const int rows = ((k1 - k0) >> 5) * 4;  // of each token
    if constexpr (kNv) {
      // E4M3 scales span 17 powers of two, so a token's blocks are scaled relative to a bound of its
      // largest magnitude: |y| <= max |x| |B|_1 |A|_1 over its blocks, multiplied in the order that y is (x by B,
      // then by A), so that it keeps fp32's range where y does.
      // Four units in flight.
      for (int q0 = warp; q0 < units; q0 += 4 * kMakerWarps) {
        float v[4][8];
        float4 br[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int q = q0 + j * kMakerWarps, st = stage_of(q), s = q - st * a.S, x = st * 32 + lane;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
          br[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (q < units && x < rows) {
            load_x8(a, s, k0 + x * 8, v[j]);
            if (a.transform) br[j] = __ldg(reinterpret_cast<const float4*>(a.B + (size_t)(k0 >> 3) * 4 + x * 4));
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int q = q0 + j * kMakerWarps;
          float m = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) m = fabsf(v[j][i]) <= 3.402823466e38f ? fmaxf(m, fabsf(v[j][i])) : m;
          if (a.transform)
            m = m * fmaxf(fmaxf(fabsf(br[j].x), fabsf(br[j].y)), fmaxf(fabsf(br[j].z), fabsf(br[j].w))) * a.a_norm;
          // (not negative: ordered as bits)
          const unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(fminf(m, 3.402823466e38f)));
          if (lane == 0 && q < units) atomicMax(&s_amax[q - stage_of(q) * a.S], bits);
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kMakers) : "memory");
      if (tid < a.S) s_xf[tid] = e8m0_value((uint32_t)(127 + digit_exponent(__uint_as_float(s_amax[tid])))) * 0.00390625f;
    }
    int pass = 0;
    for (int q = warp; q < units; q += kMakerWarps, ++pass) {
      const int st = stage_of(q), s = q - st * a.S;
      const int x = st * 32 + lane, b = lane & 3, blk = x >> 2, k = k0 + blk * 32;
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = 0.0f;
      if (x < rows) {  // (a last stage with fewer rows has zeros behind them, which no product reads)
        if (a.transform) {
          float2 u[4], y2[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float v[8];
            load_x8(a, s, k + r * 8, v);
            const float w = __ldg(a.B + (size_t)(k >> 5) * 16 + r * 4 + b);
#pragma unroll
            for (int c = 0; c < 4; ++c)
              u[c] = r == 0 ? make_float2(w * v[2 * c], w * v[2 * c + 1])
                            : fma2(make_float2(w, w), make_float2(v[2 * c], v[2 * c + 1]), u[c]);
          }
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float f = (c & 1) ? u[c >> 1].y : u[c >> 1].x;
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              const float2 m = make_float2(a.A[c * 8 + 2 * d], a.A[c * 8 + 2 * d + 1]);
              y2[d] = c == 0 ? make_float2(f * m.x, f * m.y) : fma2(make_float2(f, f), m, y2[d]);
            }
          }
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            y[2 * d] = y2[d].x;
            y[2 * d + 1] = y2[d].y;
          }
        } else {
          load_x8(a, s, k + b * 8, y);
        }
      }
      uint8_t byte;
      // The block's (NVFP4: its half's) largest magnitude; NaN and infinities win.
      unsigned top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      if constexpr (!kNv) top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const bool finite = top < 0x7F800000u;
      int e = digit_exponent(__uint_as_float(finite ? top : 0u));
      if constexpr (kNv) {
        const int e_tok = digit_exponent(__uint_as_float(s_amax[s]));
        // (y and its bound are rounded apart, so y may pass the bound's power of two by its last bits: the digits hold
        // up to 3.4 * 2^e.)
        e = min(max(e, e_tok - 17), e_tok);
        const int E = e - e_tok + 8;  // -9 .. 8: the E4M3 power of two
        byte = (uint8_t)(!finite ? 0x7F : E >= -6 ? (E + 7) << 3 : 1 << (E + 9));
      } else {
        byte = (uint8_t)(finite ? e + 127 : 255);
      }
      // (Digits of a block that is not finite are any: its scale is NaN.)
      // Fixed point: adding 1.5 * 2^23 leaves the rounded integer (at most 2^22) in the low bits, and four
      // of every digit make the digits -4 .. 3 the fields 0 .. 7.
      constexpr uint32_t kFours = 04444444444u & ((1u << (3 * kParts)) - 1);
      const float inv = e8m0_value((uint32_t)max(127 - e, 0));
      constexpr float kUnit = (float)(1 << (3 * (kParts - 1)));
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = __float_as_uint(fmaf(y[i] * inv, kUnit, 12582912.0f)) + (kFours - 0x4B400000u);
      // Two numbers to a register: of six digits the last five (15 bits) and the first, of eight four each.
      constexpr int kLow = kParts == 8 ? 4 : 5;
      uint32_t low[4], high[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        low[i] = __byte_perm(v[2 * i], v[2 * i + 1], 0x5410);
        high[i] = __byte_perm(v[2 * i] >> (3 * kLow), v[2 * i + 1] >> (3 * kLow), 0x5410);
      }
      // Column r = kP * kSp + s: kSp is a power of two above s, so the digit's part of the addresses is constant.
      uint8_t* dst = s_x + (size_t)st * (a.n * 128) + b * 4 + s * 128;
      const uint32_t turn = (uint32_t)((blk ^ s) & 7) << 4;
      // Scale byte of column r: four scale columns to a tile, row r % 32, then r / 32, then the scale column.
      const int col = kNv ? blk * 2 + (b >> 1) : blk;
      uint8_t* sc = s_sx + (col >> 2) * kSfAtom + (col & 3) + s * 16;
      const bool writes_scale = kNv ? (b & 1) == 0 : b == 0;
      for_digits<kParts>([&](auto p_tag) {
        constexpr int kP = decltype(p_tag)::value, kR = kP * kSp;
        uint32_t w;
        if constexpr (kParts - kP <= kLow)
          w = digit_codes<3 * (kParts - 1 - kP)>(low);
        else
          w = digit_codes<3 * (kParts - 1 - kP - kLow)>(high);
        *reinterpret_cast<uint32_t*>(dst + kR * 128 + (turn ^ ((kR & 7) << 4))) = w;
        if (writes_scale) sc[(kR & 31) * 16 + (kR >> 5) * 4] = byte;
      });
      fence_proxy_async_smem();  // the tensor core reads shared memory through the asynchronous proxy
      __syncwarp();
      if (lane == 0) mbar_arrive(&made[pass]);
    }
    if (lane == 0 && pass * kMakerWarps < units) mbar_arrive(&made[pass]);  // (a last pass without a unit for this warp)

    if (warp < 4) {
      // ------------------------------ epilogue ------------------------------
      const int quad = warp & 3;  // TMEM lanes 32 quad ..
      float alpha = 1.0f;
      if constexpr (kNv) alpha = a.gs != nullptr ? 1.0f / *a.gs : 1.0f;
      asm volatile("bar.sync 2, 128;" ::: "memory");  // s_xf is written
      float unit[kSp];
#pragma unroll
      for (int s = 0; s < kSp; ++s) unit[s] = kNv ? s_xf[s] : 1.0f;
      int it = 0;
      for (int tile = cluster; tile < a.tiles; tile += clusters, ++it) {
        const int buf = it & 1;
        bool ok = mbar_wait_warp(&acc_full[buf], (it >> 1) & 1);
        if (!ok) {
          if (lane == 0) set_error(a.err, kErrMmaTimeout);
          if (csize == 1) break;  // (in a cluster the four warps leave together, below)
        }
        tc_fence_after_sync();
        const uint32_t taddr = tmem + buf * a.acc_stride + ((uint32_t)(32 * quad) << 16);
        float sum[kSp];
        // The least digits first: the sum in units of the digit at hand, brought to the next one's.
        constexpr int kPiece = kSp < 8 ? kSp : 8;  // tokens at a time (registers)
#pragma unroll
        for (int s0 = 0; s0 < kSp; s0 += kPiece) {
          uint32_t v[kParts][kPiece];
#pragma unroll
          for (int p = 0; p < kParts; ++p) tmem_ld_cols<kPiece>(taddr + p * kSp + s0, v[p]);
          tmem_ld_wait();
#pragma unroll
          for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int s = 0; s < kPiece; ++s) asm volatile("" : "+r"(v[p][s]));  // not used ahead of the wait
#pragma unroll
          for (int s = 0; s < kPiece; ++s) {
            sum[s0 + s] = __uint_as_float(v[kParts - 1][s]);
#pragma unroll
            for (int p = kParts - 2; p >= 0; --p)
              sum[s0 + s] = fmaf(sum[s0 + s], 0.125f, __uint_as_float(v[p][s]));
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
#pragma unroll
        for (int s = 0; s < kSp; ++s) sum[s] *= unit[s];
        const int r = 32 * quad + lane, m = tile * kRows + r;
        auto store = [&](int s, int at, float v) {
          const size_t o = (size_t)s * a.ldo + at;
          if (a.out_bf16)
            static_cast<uint16_t*>(a.out)[o] = (uint16_t)pack_bf16x2(v * alpha, 0.0f);
          else
            static_cast<float*>(a.out)[o] = v * alpha;
        };
        if (csize == 1) {
#pragma unroll
          for (int s = 0; s < kSp; ++s)
            if (s < a.S && m < a.M) store(s, m, sum[s]);
        } else {
          // Rank c adds the rows from c * share on, rank after rank.  All four warps read the buffer, so they meet
          // after each tile: then no warp sends a tile's sums before its CTA has read the last one's.  Rank c's
          // barrier completes for a tile when every CTA's warps that hold rank c's rows have sent it, so after it
          // every CTA has read the tile before, and two buffers do.
          const int share = (kRows + (int)csize - 1) / (int)csize, mine = min(share, kRows - share * (int)crank);
          float* sums = s_sums + buf * ((kRows + 8) * kSp);
          if (ok) {
            if (tid == 0) mbar_arrive_expect_tx(&sums_ready[buf], csize * (uint32_t)(mine * kSp * 4));
            const int to = r / share;
            const uint32_t bar = mapa_shared(smem_u32(&sums_ready[buf]), (uint32_t)to);
            const uint32_t dst = mapa_shared(smem_u32(sums + ((int)crank * share + r - to * share) * kSp), (uint32_t)to);
            constexpr int kVec = kSp < 4 ? kSp : 4;
#pragma unroll
            for (int s = 0; s < kSp; s += kVec) push_cluster<kVec>(dst + s * 4, sum + s, bar);
            ok = mbar_wait_warp_cluster(&sums_ready[buf], (it >> 1) & 1);
            if (!ok && lane == 0) set_error(a.err, kErrDataTimeout);
          }
          if (ok) {
            for (int x = tid; x < mine * a.S; x += 128) {
              const int s = x / mine, row = x - s * mine, out_m = tile * kRows + (int)crank * share + row;
              float v[8];
#pragma unroll
              for (int c = 0; c < 8; ++c) v[c] = c < (int)csize ? sums[(c * share + row) * kSp + s] : 0.0f;
              float total = v[0];
#pragma unroll
              for (int c = 1; c < 8; ++c) total += v[c];
              if (out_m < a.M) store(s, out_m, total);
            }
          }
          if (!all_epilogue(ok)) break;
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (csize > 1) cluster_sync_all();  // peers may still send sums to this CTA
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

constexpr size_t kSmemLimit = 232448;

// Shared memory and TMEM of a configuration; false when it does not fit.
template <bool kNv>
bool plan(W4Args& a, int sp, int csize, size_t* smem) {
  constexpr int kAtoms = kNv ? 4 : 2;
  a.max_stages = (a.stages + csize - 1) / csize;
  a.n = (a.parts * sp + 15) & ~15;
  const size_t fixed = (size_t)a.max_stages * (a.n * 128 + kAtoms * kSfAtom) + 2 * (size_t)(kRows + 8) * sp * 4 + 32 * 4 +
                       (2 * kMaxRing + 7 + kMaxPasses) * 8 + 16 + 1024;
  a.acc_stride = (a.n + 31) & ~31;
  a.t_sx = 2 * a.acc_stride;
  a.t_sw = a.t_sx + a.max_stages * 4 * kAtoms;
  constexpr size_t kSlot = kStageBytes + kAtoms * kSfAtom;
  a.ring = kMaxRing;
  while (a.ring >= 3 && (fixed + a.ring * kSlot > kSmemLimit || a.t_sw + a.ring * 4 * kAtoms > 512)) --a.ring;
  *smem = fixed + a.ring * kSlot;
  return a.ring >= 3;
}

template <int kSp, bool kNv, int kParts>
cudaError_t launch_cfg(const LinearW4A16Launch& L, W4Args& a, cudaStream_t stream) {
  CUtensorMap tm;
  if (!make_map_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.w_codes, (uint64_t)L.N / 2, (uint64_t)L.M, (uint64_t)L.N / 2,
                   kStageK / 2, kRows, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto kern = k_linear_w4a16<kSp, kNv, kParts>;
  static PerDevice attr_set = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemLimit);
    if (e != cudaSuccess) return e;
    attr_set[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // Cluster size along K, by the time that it would take (us; fitted to sizes 1 to 8 for 1 to 16 tokens,
  // K = 512 to 12288, 1024 to 24576 out-features; its choices are 1 % above the best on average):
  //   * rounds of tiles over the clusters that run at the same time (clusters do not cross GPCs), each 0.37
  //     per stage with every SM streaming, a last one less in proportion, but 0.1; and 0.02 per CTA that
  //     exchanges sums;
  //   * the digits, 0.01 per stage, token and digit, which the CTAs of a cluster share;
  //   * 0.6 for a cluster's start.
  // Four tokens x 4096 x 24576: 14.5 us alone, 13.1 in pairs, 14.6 in threes; one x 4096 x 4096 (32
  // tiles): 6.0 in pairs, 5.7 in fours, 6.0 in eights; one x 4096 x 18944 (one tile per SM): 10.2 alone,
  // 10.9 in pairs; 16 x 4096 x 4096: 16.3 in pairs, 11.6 in fours, 10.7 in eights.
  static PerDevice active[9] = {};
  int csize = 0;
  size_t smem = 0;
  float best = 0.0f;
  for (int c = 1; c <= 8 && c <= a.stages; ++c) {
    if (!plan<kNv>(a, kSp, c, &smem)) continue;
    if (active[c][dev] == 0) {
      int n = sm_count();
      if (c > 1) {
        attr[1].val.clusterDim.x = (unsigned)c;
        cfg.gridDim = dim3((unsigned)c);
        cfg.dynamicSmemBytes = kSmemLimit;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg);
        if (e != cudaSuccess) return e;
      }
      active[c][dev] = n < 1 ? 1 : n;
    }
    const int most = active[c][dev], full = a.tiles / most, rest = a.tiles - full * most;
    float t = a.max_stages * (0.37f * full + 0.01f * a.S * kParts);
    if (rest > 0) t += a.max_stages * std::fmax(0.1f, 0.37f * rest / most);
    if (c > 1) t += 0.6f + 0.02f * c * (full + (rest > 0 ? 1 : 0));
    if (csize == 0 || t < best) {
      csize = c;
      best = t;
    }
  }
  if (csize == 0 || !plan<kNv>(a, kSp, csize, &smem)) return cudaErrorInvalidConfiguration;
  const int most = active[csize][dev], clusters = a.tiles < most ? a.tiles : most;
  attr[1].val.clusterDim.x = (unsigned)csize;
  cfg.gridDim = dim3((unsigned)(clusters * csize));
  cfg.dynamicSmemBytes = smem;
  return cudaLaunchKernelEx(&cfg, kern, tm, a);
}

template <bool kNv>
cudaError_t launch_fmt(const LinearW4A16Launch& L, cudaStream_t stream) {
  W4Args a = {};
  a.x_bf16 = L.x_bf16;
  a.N = L.N;
  a.ldx = L.ldx;
  a.transform = L.transform;
  for (int i = 0; i < 64; ++i) a.A[i] = L.A[i];
  for (int d = 0; d < 8; ++d) {
    double sum = 0.0;
    for (int c = 0; c < 8; ++c) sum += 4.0 * std::fabs(L.A[c * 8 + d]);
    a.a_norm = std::fmax(a.a_norm, (float)std::fmin(sum, (double)FLT_MAX));
  }
  a.B = L.B;
  a.scales = L.w_scales;
  a.gs = L.w_gs;
  a.M = L.M;
  a.groups = kNv ? L.N / 64 : (L.N / 32 + 3) / 4;
  a.out_bf16 = L.out_bf16;
  a.ldo = L.ldo;
  a.err = L.err;
  a.tiles = (L.M + kRows - 1) / kRows;
  a.stages = (L.N + kStageK - 1) / kStageK;
  a.parts = L.out_bf16 ? kPartsBf16 : kPartsF32;
  auto padded = [](int s) { return s <= 1 ? 1 : s <= 2 ? 2 : s <= 4 ? 4 : s <= 8 ? 8 : 16; };
  // Tokens per launch: as many as eight CTAs hold the digits of.
  int per = L.S;
  auto fits = [&](int s) {
    W4Args t = a;
    size_t smem = 0;
    for (int c = 1; c <= 8; ++c)
      if (plan<kNv>(t, padded(s), c, &smem)) return true;
    return false;
  };
  while (per > 1 && !fits(per)) per = (per + 1) / 2;
  for (int s0 = 0; s0 < L.S; s0 += per) {
    a.S = L.S - s0 < per ? L.S - s0 : per;
    a.X = static_cast<const uint8_t*>(L.X) + (size_t)s0 * L.ldx * (L.x_bf16 ? 2 : 4);
    a.out = static_cast<uint8_t*>(L.out) + (size_t)s0 * L.ldo * (L.out_bf16 ? 2 : 4);
    cudaError_t e = cudaErrorInvalidConfiguration;
    switch (padded(a.S)) {
      case 1: e = L.out_bf16 ? launch_cfg<1, kNv, kPartsBf16>(L, a, stream) : launch_cfg<1, kNv, kPartsF32>(L, a, stream); break;
      case 2: e = L.out_bf16 ? launch_cfg<2, kNv, kPartsBf16>(L, a, stream) : launch_cfg<2, kNv, kPartsF32>(L, a, stream); break;
      case 4: e = L.out_bf16 ? launch_cfg<4, kNv, kPartsBf16>(L, a, stream) : launch_cfg<4, kNv, kPartsF32>(L, a, stream); break;
      case 8: e = L.out_bf16 ? launch_cfg<8, kNv, kPartsBf16>(L, a, stream) : launch_cfg<8, kNv, kPartsF32>(L, a, stream); break;
      case 16: e = L.out_bf16 ? launch_cfg<16, kNv, kPartsBf16>(L, a, stream) : launch_cfg<16, kNv, kPartsF32>(L, a, stream); break;
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_linear_w4a16(const LinearW4A16Launch& L, cudaStream_t stream) {
  return L.nvfp4 ? launch_fmt<true>(L, stream) : launch_fmt<false>(L, stream);
}

}  // namespace batq
