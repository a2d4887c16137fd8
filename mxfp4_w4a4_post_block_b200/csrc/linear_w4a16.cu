// k_linear_w4a16: out = (X P) W'^T for 1 to 16 tokens, 4-bit prepared weights, activations kept in
// more than 16 bits (no activation quantisation).
//
//   out[s][m] = sum_c ws[m][c] * sum_{k in group c} w[m][k] y[s][k],    y_s = x_s P  (or x_s itself)
//
// with w the E2M1 codes and ws their group scales (E8M0 per 32, or E4M3 per 16 with 1 / gs on the
// result: NVFP4).  With so few tokens the weights' bytes are the work: every other choice serves to
// read them once, at full rate.
//
// Weights enter m16n8k16 matrix instructions as the 16-row operand, tokens as the 8 columns.  E2M1
// widens exactly to f16; one instruction covers 16 K of one scale group, so the scale multiplies the
// fp32 partial sum and no product is rounded.  y is normalised per token by a power of two (largest
// magnitude in [2^14, 2^15)) and enters as f16: bf16 X without a transform exactly (down to 2^-28 of
// the token's largest), anything else as two columns, f16(y) and f16(y - f16(y)), 22 bits.
//
// A unit is 32 weight rows: rows i0 .. i0 + 7 of each of the four 32-row quarters of a 128-row scale
// tile, because the tile layout holds the scales of those rows and four groups in 128 contiguous
// bytes.  The eight warps of a CTA split the unit's K in stages of 256 elements (four 8-row TMA boxes
// with the 128-byte swizzle, 4 KB, and the scales); every warp runs a ring of its own, refilled by
// itself, across units, so the stream does not stop where a unit ends.  Partial sums are added over
// the warps in shared memory, in order; when the tokens do not fit one CTA's shared memory, or when
// there are few units, the CTAs of a cluster split K and add through distributed shared memory.
#include <cmath>
#include <cstdint>

#include "host_util.h"
#include "kernels.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace batq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStageK = 256;                     // K elements per stage
constexpr int kStageBytes = 32 * kStageK / 2;    // 32 rows of codes
constexpr int kUnitRows = 32;
constexpr int kMaxStages = 4;

struct W4Args {
  const void* X;
  int x_bf16, S, N, ldx;
  int transform, split;       // split: y as two f16 columns
  float A[64], a_norm;        // a_norm: largest column sum of |A|
  const float* B;
  const uint8_t* scales;
  const float* gs;
  int M, groups;              // scale tiles per 128 rows (each 4 groups)
  int out_bf16;
  void* out;
  int ldo;
  unsigned* err;
  int units, stages, ring;    // units of 32 rows; K stages of a row; ring slots per warp
  int x_pitch;                // bytes per column of y in shared memory
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// f16 pairs of the eight E2M1 codes of a word, two codes per byte.
__device__ __forceinline__ void widen8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// 2^(b - 127) of two E8M0 bytes, as the two bf16 halves of a word (exact; 255 gives NaN).
__device__ __forceinline__ uint32_t e8m0x2(uint32_t bytes) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\t"
      "cvt.u16.u32 h, %1;\n\t"
      "cvt.rn.bf16x2.ue8m0x2 %0, h;\n\t}"
      : "=r"(r)
      : "r"(bytes));
  return r;
}

__device__ __forceinline__ uint16_t f16_bits(float v) {
  uint16_t r;
  asm("cvt.rn.f16.f32 %0, %1;" : "=h"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float f16_value(uint16_t b) {
  float r;
  asm("cvt.f32.f16 %0, %1;" : "=f"(r) : "h"(b));
  return r;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

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

// kNT: 8-column tiles of tokens.
template <int kNT, bool kNv>
__global__ void __launch_bounds__(kThreads)
    k_linear_w4a16(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ W4Args a) {
  constexpr int kTilesPerStage = kNv ? 4 : 2;     // scale tiles (four groups each) of a stage
  constexpr int kScaleBytes = kTilesPerStage * 128;
  extern __shared__ uint8_t smem_raw[];
  // (an offset, so that the compiler still knows these for shared addresses)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* s_codes = smem + (size_t)warp * a.ring * kStageBytes;
  uint8_t* s_scales = smem + (size_t)kWarps * a.ring * kStageBytes + (size_t)warp * a.ring * kScaleBytes;
  uint8_t* s_x = smem + (size_t)kWarps * a.ring * (kStageBytes + kScaleBytes);
  const int cols = a.split ? 2 * a.S : a.S;
  float* s_red = reinterpret_cast<float*>(s_x + (size_t)cols * a.x_pitch);  // [2][kWarps][kUnitRows][16]
  float* s_xf = s_red + 2 * kWarps * kUnitRows * kMaxW4A16Tokens;           // [16] 2^e of each token
  unsigned* s_amax = reinterpret_cast<unsigned*>(s_xf + 16);                // [16]
  float* s_sums = reinterpret_cast<float*>(s_amax + 16);                    // [2][kUnitRows * 16]
  uint64_t* full = reinterpret_cast<uint64_t*>(s_sums + 2 * kUnitRows * kMaxW4A16Tokens) + warp * kMaxStages;

  uint32_t csize, crank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(csize));
  asm("mov.u32 %0, %%cluster_ctaid.x;" : "=r"(crank));
  const int cluster = blockIdx.x / csize, clusters = gridDim.x / csize;
  const int st0 = (int)((long long)a.stages * crank / csize);       // this CTA's K stages
  const int st1 = (int)((long long)a.stages * (crank + 1) / csize);
  const int k0 = st0 * kStageK, k1 = min(st1 * kStageK, a.N);

  if (tid == 0) tma_prefetch_map(&tm_w);
  if (lane == 0) {
    for (int i = 0; i < a.ring; ++i) mbar_init(&full[i], 1);
    fence_barrier_init();
  }
  if (tid < 16) s_amax[tid] = 0u;
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();

  // This warp's sequence of (unit, stage): units cluster, cluster + clusters, ..; stages st0 + warp, + 8, ..
  const int per_unit = st1 - st0 > warp ? (st1 - st0 - warp + kWarps - 1) / kWarps : 0;
  int p_unit = cluster, p_i = 0, p_slot = 0;
  auto issue = [&]() {
    if (p_unit >= a.units || per_unit == 0) return;
    const int stage = st0 + warp + p_i * kWarps;
    if (lane == 0) {
      const int row0 = (p_unit >> 2) * 128 + (p_unit & 3) * 8;
      const int tiles = min(kTilesPerStage, a.groups - stage * kTilesPerStage);
      uint64_t* bar = &full[p_slot];
      mbar_arrive_expect_tx(bar, (uint32_t)(kStageBytes + tiles * 128));
#pragma unroll
      for (int q = 0; q < 4; ++q)
        tma_load_2d(s_codes + p_slot * kStageBytes + q * 1024, &tm_w, bar, stage * (kStageK / 2), row0 + q * 32);
      const uint8_t* sc = a.scales + ((size_t)(p_unit >> 2) * a.groups + (size_t)stage * kTilesPerStage) * 512 +
                          (p_unit & 3) * 128;
      for (int i = 0; i < tiles; ++i) bulk_load(s_scales + p_slot * kScaleBytes + i * 128, sc + (size_t)i * 512, 128, bar);
    }
    __syncwarp();
    if (++p_slot == a.ring) p_slot = 0;
    if (++p_i == per_unit) {
      p_i = 0;
      p_unit += clusters;
    }
  };
  for (int i = 0; i < a.ring; ++i) issue();
  __syncthreads();

  // y of this CTA's K range.  A thread makes row b (eight values) of one 4 x 8 block:
  // u = column b of B^T against the block's four rows, y = u A (A from the parameter bank).  First the
  // bound of each token's magnitudes that the normalisation needs, |y| <= max|x| * |B|_1 * |A|_1 over
  // its blocks (at most a few powers of two above the largest, out of f16's 28 spare ones).
  const int rows = ((k1 - k0) >> 5) * 4;  // of each token
  for (int s = 0; s < a.S; ++s) {
    float m = 0.0f;
    for (int x0 = tid; x0 < rows; x0 += 4 * kThreads) {
      float v[4][8];
      float4 br[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // four rows in flight
        const int x = x0 + j * kThreads;
        if (x < rows) {
          load_x8(a, s, k0 + x * 8, v[j]);
          if (a.transform) br[j] = __ldg(reinterpret_cast<const float4*>(a.B + (size_t)(k0 >> 3) * 4 + x * 4));
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (x0 + j * kThreads < rows) {
          float mj = 0.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) mj = fabsf(v[j][i]) <= 3.402823466e38f ? fmaxf(mj, fabsf(v[j][i])) : mj;
          // Row b of B bounds what x's row b adds to any y: max |B[b][.]| max |x| |A|_1, four rows together.
          if (a.transform)
            mj *= 4.0f * a.a_norm *
                  fmaxf(fmaxf(fabsf(br[j].x), fabsf(br[j].y)), fmaxf(fabsf(br[j].z), fabsf(br[j].w)));
          m = fmaxf(m, fminf(mj, 3.402823466e38f));
        }
      }
    }
    const unsigned bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m));  // non-negative: ordered like their bits
    if (lane == 0) atomicMax(&s_amax[s], bits);
  }
  __syncthreads();
  if (tid < a.S) {
    const int e = max((int)(s_amax[tid] >> 23) - 127 - 14, -126);  // the bound * 2^-e lies in [2^14, 2^15)
    s_xf[tid] = e8m0_value((uint32_t)(127 + e));
  }
  for (int s = 0; s < a.S; ++s)
  for (int x = tid; x < rows; x += kThreads) {
    const int b = x & 3, blk = x >> 2;
    const int k = k0 + blk * 32;
    const float f = e8m0_value((uint32_t)(127 - max((int)(s_amax[s] >> 23) - 127 - 14, -126)));
    float y[8];
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
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v0 = y[2 * i] * f, v1 = y[2 * i + 1] * f;
      const uint16_t h0 = f16_bits(v0), h1 = f16_bits(v1);
      hi[i] = (uint32_t)h0 | ((uint32_t)h1 << 16);
      if (a.split) {
        const uint16_t l0 = (h0 & 0x7C00u) == 0x7C00u ? 0 : f16_bits(v0 - f16_value(h0));
        const uint16_t l1 = (h1 & 0x7C00u) == 0x7C00u ? 0 : f16_bits(v1 - f16_value(h1));
        lo[i] = (uint32_t)l0 | ((uint32_t)l1 << 16);
      }
    }
    // Places in the block's 64 bytes: a lane of the products reads 16, its four elements of the first
    // instruction and its four of the second.
    uint8_t* dst = s_x + (size_t)(a.split ? 2 * s : s) * a.x_pitch + blk * 64;
    uint8_t* dlo = dst + a.x_pitch;  // columns 2 s and 2 s + 1: one lane's pair of accumulators
    if constexpr (kNv) {
      // elements 8 b ..: the groups' halves, quads 2 (b & 1) and the next, instruction b >> 1
      const int at = (b & 1) * 32 + (b >> 1) * 8;
      *reinterpret_cast<uint2*>(dst + at) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(dst + at + 16) = make_uint2(hi[2], hi[3]);
      if (a.split) {
        *reinterpret_cast<uint2*>(dlo + at) = make_uint2(lo[0], lo[1]);
        *reinterpret_cast<uint2*>(dlo + at + 16) = make_uint2(lo[2], lo[3]);
      }
    } else {
      *reinterpret_cast<uint4*>(dst + b * 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if (a.split) *reinterpret_cast<uint4*>(dlo + b * 16) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  __syncthreads();

  float alpha = 1.0f;
  if constexpr (kNv) alpha = a.gs != nullptr ? 1.0f / *a.gs : 1.0f;
  const uint8_t* xcol[kNT];
#pragma unroll
  for (int n = 0; n < kNT; ++n)  // columns behind the last repeat the first
    xcol[n] = s_x + (size_t)(n * 8 + g < cols ? n * 8 + g : 0) * a.x_pitch + t * 16;

  int slot = 0, parity = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int unit = cluster; unit < a.units; unit += clusters, parity ^= 1) {
    float acc[2][kNT][4];
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int n = 0; n < kNT; ++n) acc[q][n][0] = acc[q][n][1] = acc[q][n][2] = acc[q][n][3] = 0.0f;
    for (int i = 0; i < per_unit; ++i) {
      if (ok && !mbar_wait_warp(&full[slot], phase)) {
        if (lane == 0) set_error(a.err, kErrDataTimeout);
        ok = false;
      }
      if (!ok) break;
      const int stage = st0 + warp + i * kWarps;
      const uint8_t* codes = s_codes + slot * kStageBytes + g * 128;
      const uint8_t* scales = s_scales + slot * kScaleBytes + g * 16;
      const int nblk = min(8, (a.N >> 5) - stage * 8);
      const int xoff = (stage - st0) * (kStageK * 2);
      uint4 sc;
      uint32_t scf[4];  // MXFP4: bf16 scales of two blocks of the four row quarters
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        if (b >= nblk) break;
        if constexpr (kNv) {
          if (b % 2 == 0) sc = *reinterpret_cast<const uint4*>(scales + (b >> 1) * 128);
        } else {
          if (b % 4 == 0) sc = *reinterpret_cast<const uint4*>(scales + (b >> 2) * 128);
          if (b % 2 == 0) {
            const int sh = (b & 2) * 8;
            scf[0] = e8m0x2(sc.x >> sh);
            scf[1] = e8m0x2(sc.y >> sh);
            scf[2] = e8m0x2(sc.z >> sh);
            scf[3] = e8m0x2(sc.w >> sh);
          }
        }
        uint4 xv[kNT];
#pragma unroll
        for (int n = 0; n < kNT; ++n) xv[n] = *reinterpret_cast<const uint4*>(xcol[n] + xoff + b * 64);
        const uint8_t* at = codes + ((b ^ g) << 4);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t w0, w1;
          if constexpr (kNv) {
            // Half-words t of the block's two groups.
            const uint8_t* p0 = at + (2 * q) * 1024 + t * 2;
            const uint8_t* p1 = p0 + 1024;
            w0 = *reinterpret_cast<const uint16_t*>(p0) | ((uint32_t) * reinterpret_cast<const uint16_t*>(p0 + 8) << 16);
            w1 = *reinterpret_cast<const uint16_t*>(p1) | ((uint32_t) * reinterpret_cast<const uint16_t*>(p1 + 8) << 16);
          } else {
            w0 = *reinterpret_cast<const uint32_t*>(at + (2 * q) * 1024 + t * 4);
            w1 = *reinterpret_cast<const uint32_t*>(at + (2 * q + 1) * 1024 + t * 4);
          }
          uint32_t h0[4], h1[4];
          widen8(w0, h0);
          widen8(w1, h1);
          if constexpr (kNv) {
            const uint32_t sw0 = q == 0 ? sc.x : sc.z, sw1 = q == 0 ? sc.y : sc.w;
            const int sh = (b & 1) * 16;
            const float2 f0 = e4m3x2_values((sw0 >> sh) & 0xFFFFu), f1 = e4m3x2_values((sw1 >> sh) & 0xFFFFu);
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
              float d0[4] = {0.0f, 0.0f, 0.0f, 0.0f}, d1[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              mma_f16(d0, h0[0], h1[0], h0[1], h1[1], xv[n].x, xv[n].y);
              mma_f16(d1, h0[2], h1[2], h0[3], h1[3], xv[n].z, xv[n].w);
              acc[q][n][0] = fmaf(d1[0], f0.y, fmaf(d0[0], f0.x, acc[q][n][0]));
              acc[q][n][1] = fmaf(d1[1], f0.y, fmaf(d0[1], f0.x, acc[q][n][1]));
              acc[q][n][2] = fmaf(d1[2], f1.y, fmaf(d0[2], f1.x, acc[q][n][2]));
              acc[q][n][3] = fmaf(d1[3], f1.y, fmaf(d0[3], f1.x, acc[q][n][3]));
            }
          } else {
            const float f0 = __uint_as_float((b & 1) ? scf[2 * q] & 0xFFFF0000u : scf[2 * q] << 16);
            const float f1 = __uint_as_float((b & 1) ? scf[2 * q + 1] & 0xFFFF0000u : scf[2 * q + 1] << 16);
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
              float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              mma_f16(d, h0[0], h1[0], h0[1], h1[1], xv[n].x, xv[n].y);
              mma_f16(d, h0[2], h1[2], h0[3], h1[3], xv[n].z, xv[n].w);
              acc[q][n][0] = fmaf(d[0], f0, acc[q][n][0]);
              acc[q][n][1] = fmaf(d[1], f0, acc[q][n][1]);
              acc[q][n][2] = fmaf(d[2], f1, acc[q][n][2]);
              acc[q][n][3] = fmaf(d[3], f1, acc[q][n][3]);
            }
          }
        }
      }
      __syncwarp();  // every lane has read the slot
      if (++slot == a.ring) {
        slot = 0;
        phase ^= 1;
      }
      issue();
    }

    // Partial sums, in true units: rows q * 8 + i (quarter q), tokens.
    float* red = s_red + (size_t)parity * kWarps * kUnitRows * kMaxW4A16Tokens;
    float* mine = red + warp * kUnitRows * kMaxW4A16Tokens;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        float* lo = mine + ((2 * q) * 8 + g) * kMaxW4A16Tokens;
        float* hi = lo + 8 * kMaxW4A16Tokens;
        if (a.split) {
          const int s = n * 4 + t;
          const float f = s_xf[s];
          lo[s] = (acc[q][n][0] + acc[q][n][1]) * f;
          hi[s] = (acc[q][n][2] + acc[q][n][3]) * f;
        } else if constexpr (kNT <= 2) {
          const int s = n * 8 + 2 * t;
          const float f0 = s_xf[s], f1 = s_xf[s + 1];
          *reinterpret_cast<float2*>(lo + s) = make_float2(acc[q][n][0] * f0, acc[q][n][1] * f1);
          *reinterpret_cast<float2*>(hi + s) = make_float2(acc[q][n][2] * f0, acc[q][n][3] * f1);
        }
      }
    __syncthreads();
    // Sums over the warps, in order; thread x has row x % 32 of token x / 32.
    const int outs = kUnitRows * a.S;
    auto store = [&](int x, float sum) {
      const int r = x & 31, s = x >> 5;
      const int m = (unit >> 2) * 128 + (r >> 3) * 32 + (unit & 3) * 8 + (r & 7);
      if (m >= a.M) return;
      sum *= alpha;
      const size_t o = (size_t)s * a.ldo + m;
      if (a.out_bf16)
        static_cast<uint16_t*>(a.out)[o] = (uint16_t)pack_bf16x2(sum, 0.0f);
      else
        static_cast<float*>(a.out)[o] = sum;
    };
    float* sums = s_sums + parity * (kUnitRows * kMaxW4A16Tokens);
    for (int x = tid; x < outs; x += kThreads) {
      const float* src = red + (x & 31) * kMaxW4A16Tokens + (x >> 5);
      float v[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v[w] = src[w * kUnitRows * kMaxW4A16Tokens];
      float sum = v[0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) sum += v[w];
      if (csize > 1) sums[x] = sum; else store(x, sum);
    }
    if (csize > 1) {
      // Then over the CTAs of the cluster, in order, each taking a share of the outputs.
      cluster_sync_all();
      for (int x = tid * csize + crank; x < outs; x += kThreads * csize) {
        float v[8];
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c) v[c] = c < csize ? ld_cluster_f32(mapa_shared(smem_u32(sums + x), c)) : 0.0f;
        float sum = v[0];
#pragma unroll
        for (int c = 1; c < 8; ++c) sum += v[c];
        store(x, sum);
      }
    }
  }
  if (csize > 1) cluster_sync_all();  // peers may still read this CTA's sums
}

template <bool kNv>
size_t fixed_smem(int ring) {
  const size_t scale = kNv ? 512 : 256;
  return (size_t)kWarps * ring * (kStageBytes + scale) + 2 * kWarps * kUnitRows * kMaxW4A16Tokens * 4 + (16 + 16 + 2 * kUnitRows * kMaxW4A16Tokens) * 4 +
         kWarps * kMaxStages * 8 + 1024;
}

constexpr size_t kSmemLimit = 232448;                // one CTA per SM
constexpr size_t kSmemPair = 115200;                 // two (1 KB of each is reserved)

template <int kNT, bool kNv>
cudaError_t launch_cfg(const LinearW4A16Launch& L, W4Args& a, int cols, cudaStream_t stream) {
  // Cluster size: enough CTAs along K for the columns to fit beside a ring of two stages.
  int csize = 1;
  auto pitch = [&](int c) { return (a.stages + c - 1) / c * kStageK * 2 + 64; };
  while (csize < 8 && fixed_smem<kNv>(2) + (size_t)cols * pitch(csize) > kSmemLimit) ++csize;
  if (fixed_smem<kNv>(2) + (size_t)cols * pitch(csize) > kSmemLimit) return cudaErrorInvalidConfiguration;
  a.x_pitch = pitch(csize);
  const size_t xb = (size_t)cols * a.x_pitch;
  a.ring = 2;
  while (a.ring < kMaxStages && fixed_smem<kNv>(a.ring + 1) + xb <= kSmemPair) ++a.ring;
  const size_t smem = fixed_smem<kNv>(a.ring) + xb;
  const int per_sm = smem <= kSmemPair ? 2 : 1;

  CUtensorMap tm;
  if (!make_map_2d(&tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.w_codes, (uint64_t)L.N / 2, (uint64_t)L.M, (uint64_t)L.N / 2,
                   kStageK / 2, 8, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto kern = k_linear_w4a16<kNT, kNv>;
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
  int clusters = sm_count() * per_sm;
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
    clusters = active[dev][csize] * per_sm;
  }
  if (clusters > a.units) clusters = a.units;
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
  a.split = (L.transform || !L.x_bf16) ? 1 : 0;
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
  a.units = (L.M + 127) / 128 * 4;
  a.stages = (L.N + kStageK - 1) / kStageK;
  // Tokens per launch: as many as eight CTAs hold the columns of (all of them up to N = 16384).
  int per = L.S;
  auto fits = [&](int s) {
    const int cols = a.split ? 2 * s : s;
    return fixed_smem<kNv>(2) + (size_t)cols * ((a.stages + 7) / 8 * kStageK * 2 + 64) <= kSmemLimit;
  };
  while (per > 1 && !fits(per)) per = (per + 1) / 2;
  for (int s0 = 0; s0 < L.S; s0 += per) {
    a.S = L.S - s0 < per ? L.S - s0 : per;
    a.X = static_cast<const uint8_t*>(L.X) + (size_t)s0 * L.ldx * (L.x_bf16 ? 2 : 4);
    a.out = static_cast<uint8_t*>(L.out) + (size_t)s0 * L.ldo * (L.out_bf16 ? 2 : 4);
    const int cols = a.split ? 2 * a.S : a.S;
    const cudaError_t e = cols <= 8    ? launch_cfg<1, kNv>(L, a, cols, stream)
                          : cols <= 16 ? launch_cfg<2, kNv>(L, a, cols, stream)
                                       : launch_cfg<4, kNv>(L, a, cols, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_linear_w4a16(const LinearW4A16Launch& L, cudaStream_t stream) {
  return L.nvfp4 ? launch_fmt<true>(L, stream) : launch_fmt<false>(L, stream);
}

}  // namespace batq
