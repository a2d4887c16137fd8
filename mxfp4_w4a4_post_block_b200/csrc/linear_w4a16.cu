// k_linear_w4a16: out = (X P) W'^T for 1 to 16 tokens, 4-bit prepared weights, activations not
// quantised to the weights' width.
//
//   out[s][m] = sum_n w[m][n] y[s][n],    y_s = x_s P  (or x_s itself)
//
// with w the E2M1 codes times their group scales (E8M0 per 32, or E4M3 per 16 and 1 / gs on the
// result: NVFP4).  With so few tokens the weights' bytes are the work, so nothing is done to them:
// they go from memory by TMA straight into block-scaled 4-bit matrix instructions (kind::mxf4,
// kind::mxf4nvf4), 128 weight rows on the M side.  The tokens' precision comes from several columns
// instead of wider elements: y / scale is written as a sum of E2M1 digits,
//   r_0 = y / 2^e,  q_p = E2M1(r_p),  r_{p+1} = f_p (r_p - q_p),  f_0 = 4, f_p = 8,
// one column of the N side per token and digit, all digits of a block under the block's scale, and
// the digits' accumulators are added with the weights 1, 1/4, 1/32, .. in the epilogue.  |r_0| <= 6
// leaves a remainder of at most 1, so |r_1| <= 4, remainder at most 1/2, |r_2| <= 4 and so on: three
// bits a digit, exact arithmetic throughout.  Five digits (2^-13 of the block's largest value) serve a
// bf16 output, eight (2^-22) an fp32 one; sixteen tokens then are 80 or 128 of the 256 columns an
// instruction can have, and the tensor pipe still waits for memory.  (With the weights widened to f16 in
// registers for m16n8k16 instructions, the same products were bound by the conversions: 4 tokens x
// 4096 x 24576 took 30 us, 16 tokens 113 us.)
//
// A CTA makes its tokens' digits once, keeps them and their scales (shared memory, TMEM), and walks
// 128-row tiles of the weights: warp 0 loads stages of K = 256 (16 KB of codes by TMA with the
// 128-byte swizzle, 512-byte scale tiles) into a ring, warp 1 copies their scales into TMEM and issues
// four MMAs per stage into one of two accumulators, warps 2-5 drain the other.  When the digits do not
// fit, or when there are fewer tiles than SMs, the CTAs of a cluster split K; their sums meet in
// distributed shared memory, rank after rank.
#include <cmath>
#include <cstdint>

#include "host_util.h"
#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace batq {
namespace {

constexpr int kWarps = 10;                       // loads, MMA, 8 that make the digits (4 of them drain)
constexpr int kThreads = 32 * kWarps;
constexpr int kMakers = 32 * (kWarps - 1);       // all but the load warp make digits
constexpr int kRows = 128;                       // weight rows per tile
constexpr int kStageK = 256;                     // K elements per stage
constexpr int kStageBytes = kRows * kStageK / 2;
constexpr int kSfAtom = 512;
constexpr int kMaxRing = 10;
constexpr int kMaxParts = 8;

struct W4Args {
  const void* X;
  int x_bf16, S, N, ldx;
  int transform;
  float A[64], a_norm;        // a_norm: largest column sum of |A|
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

// Values of eight packed E2M1 codes.  (Each byte is shifted down first: taken out of one 32-bit move
// into four 8-bit registers, the upper two came back as zeros.)
__device__ __forceinline__ void e2m1x8_values(uint32_t w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b8 c;\n\t.reg .b32 hh;\n\t.reg .b16 l, h;\n\t"
        "cvt.u8.u32 c, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 hh, c;\n\t"
        "mov.b32 {l, h}, hh;\n\t"
        "cvt.f32.f16 %0, l;\n\t"
        "cvt.f32.f16 %1, h;\n\t}"
        : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
        : "r"(w >> (8 * i)));
}

// Smallest e >= -126 with a <= 6 * 2^e (6 = 1.5 * 2^2), a finite and >= 0.
__device__ __forceinline__ int digit_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  return max((int)(u >> 23) - 127 - 2 + ((u & 0x7FFFFFu) > 0x400000u ? 1 : 0), -126);
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
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

// kN consecutive fp32 columns of this thread's TMEM lane.
template <int kN>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[kN]) {
  static_assert(kN == 1 || kN == 2 || kN == 4 || kN == 8 || kN == 16, "columns");
  if constexpr (kN == 1)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r[0]) : "r"(taddr));
  else if constexpr (kN == 2)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
  else if constexpr (kN == 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
  else if constexpr (kN == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  else
    tmem_ld_16cols(taddr, r);
}

// kSp: tokens padded to a power of two (columns of a digit).
template <int kSp, bool kNv>
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
  float* s_sums = reinterpret_cast<float*>(s_sx + a.max_stages * kSfBytes);  // [2][kSp][128]
  float* s_xf = s_sums + 2 * kRows * kSp;                                  // [16] NVFP4: each token's unit
  unsigned* s_amax = reinterpret_cast<unsigned*>(s_xf + 16);               // [16]
  uint64_t* full = reinterpret_cast<uint64_t*>(s_amax + 16);
  uint64_t* empty = full + kMaxRing;
  uint64_t* acc_full = empty + kMaxRing;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* sums_ready = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sums_ready + 2);

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
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
      mbar_init(&sums_ready[i], 4 * csize);
    }
    fence_barrier_init();
  }
  if (tid < 16) s_amax[tid] = 0u;
  if (warp == 1) {
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

  if (warp == 0) {
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
  } else {
    // ------------------------------ digits ------------------------------
    // A thread makes row b (eight values) of one 4 x 8 block of one token: u = column b of B^T against
    // the block's four rows, y = u A (A from the parameter bank).
    const int id = tid - 32;
    const int rows = ((k1 - k0) >> 5) * 4;  // of each token
    if constexpr (kNv) {
      // E4M3 scales span 17 powers of two, so a token's blocks are scaled relative to a bound of its
      // largest magnitude: |y| <= max |x| |B|_1 |A|_1 over its blocks.
      for (int s = 0; s < a.S; ++s) {
        float m = 0.0f;
        for (int x0 = id; x0 < rows; x0 += 4 * kMakers) {
          float v[4][8];
          float4 br[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // four rows in flight
            const int x = x0 + j * kMakers;
            if (x < rows) {
              load_x8(a, s, k0 + x * 8, v[j]);
              if (a.transform) br[j] = __ldg(reinterpret_cast<const float4*>(a.B + (size_t)(k0 >> 3) * 4 + x * 4));
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (x0 + j * kMakers < rows) {
              float mj = 0.0f;
#pragma unroll
              for (int i = 0; i < 8; ++i) mj = fabsf(v[j][i]) <= 3.402823466e38f ? fmaxf(mj, fabsf(v[j][i])) : mj;
              if (a.transform)
                mj *= 4.0f * a.a_norm *
                      fmaxf(fmaxf(fabsf(br[j].x), fabsf(br[j].y)), fmaxf(fabsf(br[j].z), fabsf(br[j].w)));
              m = fmaxf(m, fminf(mj, 3.402823466e38f));
            }
        }
        const unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m));  // not negative: ordered as bits
        if (lane == 0) atomicMax(&s_amax[s], bits);
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kMakers) : "memory");
      if (id < a.S) s_xf[id] = e8m0_value((uint32_t)(127 + digit_exponent(__uint_as_float(s_amax[id])))) * 0.00390625f;
    }
    for (int s = 0; s < a.S; ++s) {
      int e_tok = 0;
      if constexpr (kNv) e_tok = digit_exponent(__uint_as_float(s_amax[s]));
      for (int x0 = 0; x0 < rows; x0 += kMakers) {  // (whole warps: rows of a block meet in shuffles)
        const int x = x0 + id;
        const bool live = x < rows;
        const int b = x & 3, blk = x >> 2, k = k0 + blk * 32;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.0f;
        if (live) {
          if (a.transform) {
            float u[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float v[8];
              load_x8(a, s, k + r * 8, v);
              const float w = __ldg(a.B + (size_t)(k >> 5) * 16 + r * 4 + b);
#pragma unroll
              for (int c = 0; c < 8; ++c) u[c] = r == 0 ? w * v[c] : fmaf(w, v[c], u[c]);
            }
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              y[d] = u[0] * a.A[d];
#pragma unroll
              for (int c = 1; c < 8; ++c) y[d] = fmaf(u[c], a.A[c * 8 + d], y[d]);
            }
          } else {
            load_x8(a, s, k + b * 8, y);
          }
        }
        // The block's (NVFP4: its half's) largest magnitude; NaN and infinities win.
        unsigned top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        if constexpr (!kNv) top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const bool finite = top < 0x7F800000u;
        int e = digit_exponent(__uint_as_float(finite ? top : 0u));
        if constexpr (kNv) e = max(e, e_tok - 17);
        const float inv = e8m0_value((uint32_t)max(127 - e, 0));
        uint8_t* dst = s_x + (size_t)(blk >> 3) * (a.n * 128) + b * 4;
        // Scale byte of column r: four scale columns to a tile, row r % 32, then r / 32, then the scale column.
        const int col = kNv ? blk * 2 + (b >> 1) : blk;
        uint8_t* sc = s_sx + (col >> 2) * kSfAtom + (col & 3);
        uint8_t byte;
        if constexpr (kNv) {
          const int E = e - e_tok + 8;  // -9 .. 8: the E4M3 power of two
          byte = (uint8_t)(!finite ? 0x7F : E >= -6 ? (E + 7) << 3 : 1 << (E + 9));
        } else {
          byte = (uint8_t)(finite ? e + 127 : 255);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = finite ? y[i] * inv : 0.0f;
        if (live) {
          float f = 4.0f;
          for (int p = 0; p < a.parts; ++p) {
            const int r = p * kSp + s;
            const uint32_t w = e2m1x8(y[0], y[1], y[2], y[3], y[4], y[5], y[6], y[7]);
            *reinterpret_cast<uint32_t*>(dst + r * 128 + (((blk & 7) ^ (r & 7)) << 4)) = w;
            if (kNv ? (b & 1) == 0 : b == 0) sc[(r & 31) * 16 + (r >> 5) * 4] = byte;
            float q[8];
            e2m1x8_values(w, q);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = (y[i] - q[i]) * f;
            f = 8.0f;
          }
        }
      }
    }
    fence_proxy_async_smem();  // the tensor core reads shared memory through the asynchronous proxy
    asm volatile("bar.sync 1, %0;" ::"n"(kMakers) : "memory");

    if (warp == 1) {
      // ------------------------------ MMA issuer ------------------------------
      // The whole warp runs the loop (warp-uniform state); one elected lane issues.
      const bool issuer = elect_one();
      tc_fence_after_sync();
      if (issuer) {
        for (int i = 0; i < (st1 - st0) * kAtoms; ++i)
          tc_cp_32x128b_warpx4(tmem + a.t_sx + 4 * i, sdesc_sf_atom(smem_u32(s_sx + i * kSfAtom)));
      }
      __syncwarp();
      int s = 0, it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = cluster; tile < a.tiles && ok; tile += clusters, ++it) {
        const int buf = it & 1;
        if (!mbar_wait_warp(&acc_empty[buf], ((it >> 1) & 1) ^ 1)) {
          if (issuer) set_error(a.err, kErrDrainTimeout);
          break;
        }
        tc_fence_after_sync();
        const uint32_t t_acc = tmem + buf * a.acc_stride;
        for (int st = st0; st < st1; ++st) {
          if (!mbar_wait_warp(&full[s], ph)) {
            if (issuer) set_error(a.err, kErrDataTimeout);
            ok = false;
            break;
          }
          tc_fence_after_sync();
          if (issuer) {
            const int nmma = min(4, (a.N - st * kStageK) >> 6);
            const int atoms = kNv ? nmma : (nmma + 1) >> 1;
            const uint64_t dsw = sdesc_sf_atom(smem_u32(s_sw + s * kSfBytes));
            const uint32_t tsw = tmem + a.t_sw + s * (4 * kAtoms);
            const uint32_t tsx = tmem + a.t_sx + (st - st0) * (4 * kAtoms);
            // Copies and MMAs of one thread run in order.
            for (int i = 0; i < atoms; ++i) tc_cp_32x128b_warpx4(tsw + 4 * i, dsw + (uint64_t)(i * (kSfAtom >> 4)));
            const uint64_t dw = sdesc_kmajor_sw128(smem_u32(s_w + s * kStageBytes));
            const uint64_t dx = sdesc_kmajor_sw128(smem_u32(s_x + (size_t)(st - st0) * (a.n * 128)));
            for (int j = 0; j < nmma; ++j) {
              const uint32_t acc = (st > st0 || j > 0) ? 1u : 0u;
              if constexpr (kNv)
                tc_mma_nvf4(t_acc, dw + (uint64_t)(j * 2), dx + (uint64_t)(j * 2), idesc_nvf4(kRows, a.n), tsw + 4 * j,
                            tsx + 4 * j, acc);
              else
                tc_mma_mxf4(t_acc, dw + (uint64_t)(j * 2), dx + (uint64_t)(j * 2),
                            idesc_mxf4(a.n, (2 * j) & 3, (2 * j) & 3), tsw + 4 * (j >> 1), tsx + 4 * (j >> 1), acc);
            }
            tc_commit(&empty[s]);
            if (st == st1 - 1) tc_commit(&acc_full[buf]);
          }
          __syncwarp();
          if (++s == a.ring) {
            s = 0;
            ph ^= 1;
          }
        }
      }
    } else if (warp < 6) {
      // ------------------------------ epilogue ------------------------------
      const int quad = warp & 3;  // TMEM lanes 32 quad ..
      float alpha = 1.0f;
      if constexpr (kNv) alpha = a.gs != nullptr ? 1.0f / *a.gs : 1.0f;
      float unit[kSp];
#pragma unroll
      for (int s = 0; s < kSp; ++s) unit[s] = kNv ? s_xf[s] : 1.0f;
      int it = 0;
      for (int tile = cluster; tile < a.tiles; tile += clusters, ++it) {
        const int buf = it & 1;
        if (!mbar_wait_warp(&acc_full[buf], (it >> 1) & 1)) {
          if (lane == 0) set_error(a.err, kErrMmaTimeout);
          break;
        }
        tc_fence_after_sync();
        const uint32_t taddr = tmem + buf * a.acc_stride + ((uint32_t)(32 * quad) << 16);
        float sum[kSp];
        float f = 1.0f;
        for (int p = 0; p < a.parts; ++p) {
          uint32_t v[kSp];
          tmem_ld_cols<kSp>(taddr + p * kSp, v);
          tmem_ld_wait();
#pragma unroll
          for (int s = 0; s < kSp; ++s) asm volatile("" : "+r"(v[s]));  // not used ahead of the wait
#pragma unroll
          for (int s = 0; s < kSp; ++s) sum[s] = p == 0 ? __uint_as_float(v[s]) : fmaf(__uint_as_float(v[s]), f, sum[s]);
          f *= p == 0 ? 0.25f : 0.125f;
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[buf]);
#pragma unroll
        for (int s = 0; s < kSp; ++s) sum[s] *= unit[s];
        const int r = 32 * quad + lane, m = tile * kRows + r;
        auto store = [&](int s, float v) {
          const size_t o = (size_t)s * a.ldo + m;
          if (a.out_bf16)
            static_cast<uint16_t*>(a.out)[o] = (uint16_t)pack_bf16x2(v * alpha, 0.0f);
          else
            static_cast<float*>(a.out)[o] = v * alpha;
        };
        if (csize == 1) {
#pragma unroll
          for (int s = 0; s < kSp; ++s)
            if (s < a.S && m < a.M) store(s, sum[s]);
        } else {
          float* sums = s_sums + buf * (kRows * kSp);
#pragma unroll
          for (int s = 0; s < kSp; ++s) sums[s * kRows + r] = sum[s];
          __syncwarp();
          if (lane == 0)
            for (uint32_t c = 0; c < csize; ++c) mbar_arrive_release_cluster(mapa_shared(smem_u32(&sums_ready[buf]), c));
          if (!mbar_wait_warp_cluster(&sums_ready[buf], (it >> 1) & 1)) {
            if (lane == 0) set_error(a.err, kErrDataTimeout);
            break;
          }
          // Rank c adds and writes every csize-th token's row, rank after rank.
          for (int s = (int)crank; s < a.S; s += (int)csize) {
            float v[8];
#pragma unroll
            for (uint32_t c = 0; c < 8; ++c)
              v[c] = c < csize ? ld_cluster_f32(mapa_shared(smem_u32(sums + s * kRows + r), c)) : 0.0f;
            float total = v[0];
#pragma unroll
            for (int c = 1; c < 8; ++c) total += v[c];
            if (m < a.M) store(s, total);
          }
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncthreads();
  if (csize > 1) cluster_sync_all();  // peers may still read this CTA's sums
  if (warp == 1) {
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
  const size_t fixed = (size_t)a.max_stages * (a.n * 128 + kAtoms * kSfAtom) + 2 * (size_t)kRows * sp * 4 + 32 * 4 +
                       (2 * kMaxRing + 6) * 8 + 16 + 1024;
  a.acc_stride = (a.n + 31) & ~31;
  a.t_sx = 2 * a.acc_stride;
  a.t_sw = a.t_sx + a.max_stages * 4 * kAtoms;
  constexpr size_t kSlot = kStageBytes + kAtoms * kSfAtom;
  a.ring = kMaxRing;
  while (a.ring >= 3 && (fixed + a.ring * kSlot > kSmemLimit || a.t_sw + a.ring * 4 * kAtoms > 512)) --a.ring;
  *smem = fixed + a.ring * kSlot;
  return a.ring >= 3;
}

template <int kSp, bool kNv>
cudaError_t launch_cfg(const LinearW4A16Launch& L, W4Args& a, cudaStream_t stream) {
  // Cluster size along K: until the digits fit beside a ring of three stages; then, with fewer tiles
  // than half of the SMs, while more SMs can take part with two stages or more each.
  size_t smem = 0;
  int csize = 1;
  while (csize <= 8 && !plan<kNv>(a, kSp, csize, &smem)) ++csize;
  if (csize > 8) return cudaErrorInvalidConfiguration;
  while (csize * 2 <= 8 && a.tiles * csize * 2 <= sm_count() && a.stages >= csize * 4) csize *= 2;
  if (!plan<kNv>(a, kSp, csize, &smem)) return cudaErrorInvalidConfiguration;

  CUtensorMap tm;
  if (!make_map_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.w_codes, (uint64_t)L.N / 2, (uint64_t)L.M, (uint64_t)L.N / 2,
                   kStageK / 2, kRows, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto kern = k_linear_w4a16<kSp, kNv>;
  static bool attr_set[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemLimit);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)csize;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  // As many clusters as run at the same time (clusters do not cross GPCs, so fewer than SMs / size).
  int clusters = sm_count();
  if (csize > 1) {
    static int active[64][9] = {};
    if (active[dev][csize] == 0) {
      cfg.gridDim = dim3((unsigned)csize);
      cudaLaunchConfig_t one = cfg;
      one.dynamicSmemBytes = kSmemLimit;
      int n = 0;
      cudaError_t e = cudaOccupancyMaxActiveClusters(&n, kern, &one);
      if (e != cudaSuccess) return e;
      active[dev][csize] = n < 1 ? 1 : n;
    }
    clusters = active[dev][csize];
  }
  if (clusters > a.tiles) clusters = a.tiles;
  cfg.gridDim = dim3((unsigned)(clusters * csize));
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
    float sum = 0.0f;
    for (int c = 0; c < 8; ++c) sum += std::fabs(L.A[c * 8 + d]);
    a.a_norm = sum > a.a_norm ? sum : a.a_norm;
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
  a.parts = L.out_bf16 ? 5 : kMaxParts;
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
      case 1: e = launch_cfg<1, kNv>(L, a, stream); break;
      case 2: e = launch_cfg<2, kNv>(L, a, stream); break;
      case 4: e = launch_cfg<4, kNv>(L, a, stream); break;
      case 8: e = launch_cfg<8, kNv>(L, a, stream); break;
      case 16: e = launch_cfg<16, kNv>(L, a, stream); break;
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
