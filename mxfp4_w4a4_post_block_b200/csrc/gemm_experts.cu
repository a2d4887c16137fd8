// k_gemm_experts: MXFP4 x MXFP4 products of ragged row groups, one weight matrix per group (experts).
//
//   out[r][m] = sum_n deq(a)[r][n] deq(w_e)[m][n]   for r in [offsets[e], offsets[e + 1])
//
// The offsets are on the device, so the list of tiles is made there: every CTA scans the E counts
// into shared memory and the persistent CTA pairs walk the same list (expert, token tile, weight
// tile).  A tile is 256 weight rows (the M side of cta_group::2: 128 per CTA, always full) by up to
// 256 tokens on the N side, whose size is chosen per tile in steps of 16: with tokens on the M side a
// group of 300 rows would cost 512, here 304.  The groups' tokens are split evenly over their tiles.
//
// The roles and the pipeline are those of the pair GEMM for one matrix (gemm_pair.cu): warp 0 loads
// codes and weight scales by TMA into three 66 KB stages of K = 512, warp 10 of the leader copies the
// scales into TMEM, warp 1 issues the MMAs, eight epilogue warps drain the accumulator.  What is
// different is the token side's scales: a group starts at any row, while the tensor cores want 128-row
// x 4-column tiles, so they come in the LINEAR layout and five warps per CTA re-tile them: each lane
// reads the 16 scale bytes of rows l, l + 32, .. of the tile and writes the tiles with one 16-byte
// store per atom.  The leader's copies read both CTAs' shared memory, so the peer's warps publish theirs
// with a cluster-scope release, which takes about as long as the operand loads in flight; the scales
// therefore have a ring of their own and run up to five stages ahead.  (In the stages' ring, 16384
// rows of 8 experts took 169 us.)
//
// Epilogue: a lane holds one weight row, a register one token; pairs of tokens are exchanged between
// neighbouring lanes so that a store writes two consecutive out-features of one token (64
// contiguous bytes per token and warp).  Rows outside every group are not written.
//
// Measured: 16384 rows of 8 experts, 4096 x 4096: 131 us (4.2 PFLOP/s) in a short row of calls, 152 to 157 us
// (3.5 PFLOP/s) in a long one, bound by the tensor pipe with the
// scale copies in its queue and by one accumulator; 8190 rows of 128 experts, 2112 x 1040: 47 us, 64 rows
// of 64, 4096 x 2048: 33 us, bound by memory and by stages and tiles that are nearly empty but take as
// long as whole ones (stages of K = 256: 57 and 42 us).
#include <cstdint>

#include "host_util.h"
#include "kernels.h"
#include "ptx.cuh"

namespace batq {
namespace {

constexpr int kRowsPerCta = 128;
constexpr int kTileM = 256;             // weight rows per pair
constexpr int kTileN = 256;             // most tokens per tile
constexpr int kStages = 3;
constexpr int kBK = 512;                // K elements per stage
constexpr int kSwTile = 128 * 128;      // 128 rows x 128 bytes
constexpr int kWBytes = 2 * kSwTile;    // own weight rows
constexpr int kXBytes = 2 * kSwTile;    // own half of the tokens
constexpr int kSfAtom = 512;
constexpr int kAtoms = 4;               // 4-scale atoms per row and stage
constexpr int kSfwBytes = kAtoms * kSfAtom;
constexpr int kSfxBytes = 2 * kAtoms * kSfAtom;
constexpr int kStageBytes = kWBytes + kXBytes + kSfwBytes;
constexpr int kSxSlots = 5;             // ring of the token scales, made up to five stages ahead
constexpr int kEpiWarps = 8;
constexpr int kSfWarp = 2 + kEpiWarps;
constexpr int kSxWarp = kSfWarp + 1;    // first of the warps that re-tile the token scales
constexpr int kSxWarps = 5;
constexpr int kThreads = (kSxWarp + kSxWarps) * 32;
constexpr int kTmemCols = 512;
constexpr int kSfwCols = 4 * kAtoms, kSfxCols = 8 * kAtoms;
constexpr int kListBytes = (3 * kMaxExperts + 4) * 4;  // per expert: first row, rows, first tile
constexpr int kSxOffset = kStages * kStageBytes;
constexpr int kListOffset = kSxOffset + kSxSlots * kSfxBytes;
constexpr int kBarOffset = kListOffset + kListBytes;
constexpr int kSmemBytes = kBarOffset + 256 + 1024;
static_assert(kStageBytes % 1024 == 0 && kListBytes % 16 == 0, "alignment");
static_assert(kTileN + kStages * (kSfwCols + kSfxCols) <= kTmemCols, "TMEM budget");
static_assert(kSmemBytes <= 232448, "shared memory budget");

struct ExpertsArgs {
  const int* offsets;
  const uint8_t* a_scales;
  int E, T, M, N, k;       // k: scale columns of the activations (N / 32)
  int tiles_m;             // 256-row weight tiles per expert
  int w_row_tiles;         // 128-row scale tiles per expert
  int num_kstages;
  int sf_box_chunks;
  void* out;
  int ldo;
  unsigned* err;
};

// One tile of the list.
struct Tile {
  int e, w_row;            // expert, first weight row
  int row, count, n;       // first token row, tokens, N of the MMA (count rounded up to 16)
};

__device__ __forceinline__ Tile tile_of(const ExpertsArgs& a, const int* s_off, const int* s_unit, int u) {
  int lo = 0, hi = a.E;  // the last expert with s_unit[e] <= u
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_unit[mid] <= u) lo = mid; else hi = mid;
  }
  Tile t;
  t.e = lo;
  const int cnt = s_off[2 * lo + 1], at = u - s_unit[lo];
  const int tiles_n = (cnt + kTileN - 1) / kTileN;
  const int size = ((cnt + tiles_n - 1) / tiles_n + 15) & ~15;
  const int tn = at / a.tiles_m;
  t.w_row = (at % a.tiles_m) * kTileM;
  t.row = s_off[2 * lo] + tn * size;
  t.count = min(size, cnt - tn * size);
  t.n = (t.count + 15) & ~15;
  return t;
}

__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait_acquire_cluster(uint64_t* bar, uint32_t parity, uint32_t hint_ns) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity), "r"(hint_ns)
      : "memory");
  return done != 0;
}

// mbar_wait_warp with an acquire at cluster scope.
__device__ __forceinline__ bool mbar_wait_warp_cluster(uint64_t* bar, uint32_t parity) {
  bool ok = true;
  if (!mbar_try_wait_acquire_cluster(bar, parity, kSuspendHintNs)) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait_acquire_cluster(bar, parity, kSuspendHintNs)) {
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        ok = false;
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok) != 0;
}

template <bool kOutBF16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_gemm_experts(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_sfw,
                   const __grid_constant__ CUtensorMap tm_x8, const __grid_constant__ CUtensorMap tm_x32,
                   const ExpertsArgs a) {
  extern __shared__ uint8_t smem_raw[];
  // (an offset, so that the compiler still knows these for shared addresses)
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  int* s_off = reinterpret_cast<int*>(smem + kListOffset);             // [E] {first row, rows}
  int* s_unit = s_off + 2 * kMaxExperts;                              // [E + 1] first tile of each expert
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOffset);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 1;
  uint64_t* sf_ready = acc_empty + 1;  // [kStages], leader only
  uint64_t* sx_full = sf_ready + kStages;  // [kSxSlots], leader only
  uint64_t* sx_empty = sx_full + kSxSlots;
  uint64_t* all_done = sx_empty + kSxSlots;  // products and scale copies have ended, leader only
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(all_done + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = (rank == 0);
  const int cluster_id = blockIdx.x >> 1, num_clusters = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    tma_prefetch_map(&tm_w);
    tma_prefetch_map(&tm_sfw);
    tma_prefetch_map(&tm_x8);
    tma_prefetch_map(&tm_x32);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sf_ready[s], 1);
    }
    for (int s = 0; s < kSxSlots; ++s) {
      mbar_init(&sx_full[s], 2);  // both CTAs' token scales
      mbar_init(&sx_empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 2 * kEpiWarps);
    mbar_init(all_done, 2);
    fence_barrier_init();
    griddep_launch_dependents();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, kTmemCols);
    tmem_relinquish_pair();
  }
  // The list of tiles (the offsets may come from the preceding grid).
  griddep_wait();
  if (warp == 0) {
    // Offsets count as at least the ones before them and inside [0, T], so no row has two experts.
    int before = 0, reached = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      int begin = e <= a.E ? min(max(a.offsets[e], 0), a.T) : 0;
      int end = e < a.E ? min(max(a.offsets[e + 1], 0), a.T) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, begin, o);
        if (lane >= o) begin = max(begin, x);
      }
      begin = max(begin, reached);
      end = max(end, begin);
      reached = __shfl_sync(0xffffffffu, max(begin, end), 31);
      const int cnt = e < a.E ? end - begin : 0;
      const int n = (cnt + kTileN - 1) / kTileN * a.tiles_m;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (e < a.E) {
        s_off[2 * e] = begin;
        s_off[2 * e + 1] = cnt;
        s_unit[e] = before + incl - n;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_unit[a.E] = before;
  }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // barriers of both CTAs initialised, TMEM allocated in both
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;
  const uint32_t t_acc = tmem, t_sfw = tmem + kTileN, t_sfx = t_sfw + kStages * kSfwCols;
  const int num_units = s_unit[a.E];
  const int nks = a.num_kstages;

  // Every role walks this pair's tiles and their K stages in the same order.
  if (warp == 0) {
    // ------------------------------ loads (both CTAs) ------------------------------
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = cluster_id; u < num_units && ok; u += num_clusters) {
        const Tile t = tile_of(a, s_off, s_unit, u);
        const int half = t.n >> 1;                       // tokens of each CTA
        const int x0 = t.row + (int)rank * half;
        // Boxes of 8 rows for a few tokens, of 32 otherwise; rows behind the tile's are loaded and not used.
        const int step = half <= 16 ? 8 : 32, boxes = (half + step - 1) / step;
        const uint32_t tx = (uint32_t)(kWBytes + boxes * step * 256 + a.sf_box_chunks * 256);
        const int wsf = t.e * a.w_row_tiles + min(t.w_row / kRowsPerCta + (int)rank, a.w_row_tiles - 1);
        for (int ks = 0; ks < nks; ++ks) {
          if (!mbar_wait(&empty[s], ph ^ 1)) {
            set_error(a.err, kErrReleaseTimeout);
            ok = false;
            break;
          }
          uint8_t* st = smem + s * kStageBytes;
          const uint32_t bar = mapa_shared(smem_u32(&full[s]), 0);
          if (leader) mbar_arrive_expect_tx(&full[s], 2u * tx);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            tma_load_3d_pair(st + h * kSwTile, &tm_w, bar, ks * 256 + h * 128, t.w_row + (int)rank * kRowsPerCta, t.e);
          for (int b = 0; b < boxes; ++b) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint8_t* dst = st + kWBytes + h * kSwTile + b * step * 128;
              tma_load_2d_pair(dst, step == 8 ? &tm_x8 : &tm_x32, bar, ks * 256 + h * 128, x0 + b * step);
            }
          }
          tma_load_3d_pair(st + kWBytes + kXBytes, &tm_sfw, bar, 0, ks * 2 * kAtoms, wsf);
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
    }
  } else if (warp >= kSxWarp) {
    // ---------------------- token scales (both CTAs): every kSxWarps-th stage ----------------------
    const int turn = warp - kSxWarp;
    int stage = 0;          // running stage number
    bool ok = true;
    for (int u = cluster_id; u < num_units && ok; u += num_clusters) {
      const Tile t = tile_of(a, s_off, s_unit, u);
      const int groups = (t.n + 31) >> 5;  // 32-row groups
      for (int ks = 0; ks < nks; ++ks, ++stage) {
        if (stage % kSxWarps != turn) continue;
        const int c0 = ks * 16;
        uint32_t v[8][4];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[q][0] = v[q][1] = v[q][2] = v[q][3] = 0;
          const int r = q * 32 + lane;
          if (q < groups && r < t.count) {
            const uint8_t* src = a.a_scales + (size_t)(t.row + r) * a.k + c0;
            if ((a.k & 15) == 0) {
              const uint4 w = *reinterpret_cast<const uint4*>(src);
              v[q][0] = w.x; v[q][1] = w.y; v[q][2] = w.z; v[q][3] = w.w;
            } else if ((a.k & 3) == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (c0 + 4 * i < a.k) v[q][i] = *reinterpret_cast<const uint32_t*>(src + 4 * i);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (c0 + 2 * i < a.k)
                  v[q][i >> 1] |= (uint32_t) * reinterpret_cast<const uint16_t*>(src + 2 * i) << ((i & 1) * 16);
            }
          }
        }
        const int slot = stage % kSxSlots;
        if (!mbar_wait_warp(&sx_empty[slot], ((stage / kSxSlots) & 1) ^ 1)) {
          if (lane == 0) set_error(a.err, kErrReleaseTimeout);
          ok = false;
          break;
        }
        uint8_t* dst = smem + kSxOffset + slot * kSfxBytes;
        // Atom x of the row tile R: row r at 16 (r % 32), its 32-row quarter's four bytes beside each other.
#pragma unroll
        for (int R = 0; R < 2; ++R)
          if (4 * R < groups)
#pragma unroll
            for (int x = 0; x < kAtoms; ++x)
              *reinterpret_cast<uint4*>(dst + (R * kAtoms + x) * kSfAtom + lane * 16) =
                  make_uint4(v[4 * R][x], v[4 * R + 1][x], v[4 * R + 2][x], v[4 * R + 3][x]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (leader)
            mbar_arrive(&sx_full[slot]);
          else
            mbar_arrive_release_cluster(mapa_shared(smem_u32(&sx_full[slot]), 0));
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer (leader only) ------------------------------
    if (leader) {
      const bool issuer = elect_one();
      int s = 0;
      uint32_t ph = 0, iter = 0;
      bool ok = true;
      for (int u = cluster_id; u < num_units && ok; u += num_clusters, ++iter) {
        const int n = tile_of(a, s_off, s_unit, u).n;
        for (int ks = 0; ks < nks; ++ks) {
          if (ks == 0) {
            if (!mbar_wait_warp(acc_empty, (iter & 1) ^ 1)) {
              if (issuer) set_error(a.err, kErrDrainTimeout);
              ok = false;
              break;
            }
            tc_fence_after_sync();
          }
          if (!mbar_wait_warp(&sf_ready[s], ph)) {
            if (issuer) set_error(a.err, kErrDataTimeout);
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint64_t dw = sdesc_kmajor_sw128(smem_u32(smem + s * kStageBytes));
          const uint64_t dx = dw + (uint64_t)(kWBytes >> 4);
          const uint32_t tw = t_sfw + s * kSfwCols, tx = t_sfx + s * kSfxCols;
          const int nmma = min(8, (a.N - ks * kBK) >> 6);
          if (issuer) {
            for (int j = 0; j < nmma; ++j) {
              const uint64_t off = (uint64_t)((j >> 2) * (kSwTile >> 4) + (j & 3) * 2);
              const int sf_id = (2 * j) & 3;
              tc_mma_pair_mxf4(t_acc, dw + off, dx + off, idesc_mxf4_m256(n, sf_id, sf_id), tw + (j >> 1) * 4,
                               tx + (j >> 1) * 8, (ks > 0 || j > 0) ? 1u : 0u);
            }
            tc_commit_pair(&empty[s], 0x3);
            if (ks == nks - 1) tc_commit_pair(acc_full, 0x3);
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // All instructions have ended before TMEM is freed, given up or not.
      if (issuer) tc_commit_pair_local(all_done);
      __syncwarp();
      if (!mbar_wait_warp(all_done, 0) && issuer) set_error(a.err, kErrMmaTimeout);
      // Where any role gave up this one does too, and copies may be on their way (of both CTAs, on the leader's barriers):
      // each stage's barrier gets its time, in the phase that it is in.
      for (int i = 0; !ok && i < 2 * kStages; ++i) mbar_wait_warp(&full[i >> 1], i & 1);
    }
  } else if (warp == kSfWarp) {
    // ---------------------- scale copies into TMEM (leader only) ----------------------
    if (leader) {
      const bool issuer = elect_one();
      int s = 0, x_slot = 0;
      uint32_t ph = 0, x_ph = 0;
      bool ok = true;
      for (int u = cluster_id; u < num_units && ok; u += num_clusters) {
        const int n = tile_of(a, s_off, s_unit, u).n;
        for (int ks = 0; ks < nks; ++ks) {
          if (!mbar_wait_warp_cluster(&sx_full[x_slot], x_ph) || !mbar_wait_warp(&full[s], ph)) {
            if (issuer) set_error(a.err, kErrDataTimeout);
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const int nmma = min(8, (a.N - ks * kBK) >> 6);
          const int atoms = (nmma + 1) >> 1;
          const uint64_t dw = sdesc_sf_atom(smem_u32(smem + s * kStageBytes) + kWBytes + kXBytes);
          const uint64_t dx = sdesc_sf_atom(smem_u32(smem + kSxOffset + x_slot * kSfxBytes));
          const uint32_t tw = t_sfw + s * kSfwCols, tx = t_sfx + s * kSfxCols;
          if (issuer) {
            for (int x = 0; x < atoms; ++x) {
              const uint64_t off = (uint64_t)(x * (kSfAtom >> 4));
              tc_cp_pair_32x128b_warpx4(tw + x * 4, dw + off);
              tc_cp_pair_32x128b_warpx4(tx + x * 8, dx + off);
              if (n > 128) tc_cp_pair_32x128b_warpx4(tx + x * 8 + 4, dx + (uint64_t)((kAtoms * kSfAtom) >> 4) + off);
            }
            tc_commit_pair_local(&sf_ready[s]);
            tc_commit_pair(&sx_empty[x_slot], 0x3);
          }
          __syncwarp();
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
          if (++x_slot == kSxSlots) {
            x_slot = 0;
            x_ph ^= 1;
          }
        }
      }
      if (issuer) tc_commit_pair_local(all_done);
      __syncwarp();
    }
  } else {
    // ------------------------------ epilogue (both CTAs) ------------------------------
    const int ew = warp - 2, quad = warp & 3;
    const uint32_t acc_empty_leader = mapa_shared(smem_u32(acc_empty), 0);
    uint32_t iter = 0;
    for (int u = cluster_id; u < num_units; u += num_clusters, ++iter) {
      const Tile t = tile_of(a, s_off, s_unit, u);
      const int wcols = ((t.n >> 1) + 31) & ~31;      // tokens of this warp's half, a multiple of 32
      const int col0 = (ew >> 2) * wcols;
      if (!mbar_wait_warp(acc_full, iter & 1)) {
        if (lane == 0) set_error(a.err, kErrMmaTimeout);
        break;
      }
      tc_fence_after_sync();
      const uint32_t taddr = t_acc + ((uint32_t)(32 * quad) << 16) + col0;
      const int m = t.w_row + (int)rank * kRowsPerCta + 32 * quad + lane;
      const bool m_ok = m < a.M;  // M is a multiple of 16: neighbouring lanes agree
      const int left = min(t.count - col0, wcols);
      auto release = [&]() {
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(acc_empty_leader);
      };
      // (16 warps have 128 registers each: bf16 holds all of its 128 columns as pairs, fp32 64 at a time.)
      if constexpr (kOutBF16) {
        uint32_t v[4][16];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (32 * c < wcols) {
            uint32_t w[32];
            tmem_ld_32cols(taddr + 32 * c, w);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(w[i]));  // not used ahead of the wait
#pragma unroll
            for (int i = 0; i < 16; ++i) v[c][i] = pack_bf16x2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
          }
        release();
        uint16_t* o = static_cast<uint16_t*>(a.out) + (size_t)(t.row + col0 + (lane & 1)) * a.ldo + (m & ~1);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (32 * c >= left) break;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const uint32_t r = v[c][i / 2];
            const uint32_t p = __shfl_xor_sync(0xffffffffu, r, 1);
            const uint32_t x = (lane & 1) ? __byte_perm(p, r, 0x7632) : __byte_perm(r, p, 0x5410);
            if (m_ok && 32 * c + i + (lane & 1) < left) *reinterpret_cast<uint32_t*>(o + (size_t)(32 * c + i) * a.ldo) = x;
          }
        }
      } else {
        float* o = static_cast<float*>(a.out) + (size_t)(t.row + col0) * a.ldo + m;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[2][32];
#pragma unroll
          for (int c = 0; c < 2; ++c)
            if (64 * h + 32 * c < wcols) tmem_ld_32cols(taddr + 64 * h + 32 * c, w[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(w[c][i]));
          if (h == 1) release();
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (64 * h + 32 * c >= left) break;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (m_ok && 64 * h + 32 * c + i < left) o[(size_t)(64 * h + 32 * c + i) * a.ldo] = __uint_as_float(w[c][i]);
          }
        }
      }
    }
  }

  tc_fence_before_sync();
  __syncwarp();
  cluster_sync_all();  // all MMAs done and all TMEM reads finished in both CTAs
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

template <bool kOutBF16>
cudaError_t launch_impl(const ExpertsLaunch& L, cudaStream_t stream) {
  CUtensorMap tm_w, tm_sfw, tm_x8, tm_x32;
  const uint64_t row_bytes = (uint64_t)L.N / 2;
  const uint64_t chunks = (uint64_t)((L.N / 32 + 3) / 4) * 2;  // 256-byte chunks of a row tile's scales
  const uint64_t w_row_tiles = (uint64_t)(L.M + 127) / 128;
  const int box_chunks = (int)(chunks < 2 * kAtoms ? chunks : 2 * kAtoms);
  if (!make_map_3d_swizzled(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.w_codes, row_bytes, (uint64_t)L.M, (uint64_t)L.E,
                            row_bytes, row_bytes * L.M, 128, kRowsPerCta, 1, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_3d(&tm_sfw, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.w_scales, 256, chunks, w_row_tiles * L.E, 256,
                   chunks * 256, 256, box_chunks, 1) ||
      !make_map_2d(&tm_x8, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.a_codes, row_bytes, (uint64_t)L.T, row_bytes, 128, 8,
                   CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_2d(&tm_x32, CU_TENSOR_MAP_DATA_TYPE_UINT8, L.a_codes, row_bytes, (uint64_t)L.T, row_bytes, 128, 32,
                   CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  ExpertsArgs a = {};
  a.offsets = L.offsets;
  a.a_scales = L.a_scales;
  a.E = L.E;
  a.T = L.T;
  a.M = L.M;
  a.N = L.N;
  a.k = L.N / 32;
  a.tiles_m = (L.M + kTileM - 1) / kTileM;
  a.w_row_tiles = (int)w_row_tiles;
  a.num_kstages = (L.N + kBK - 1) / kBK;
  a.sf_box_chunks = box_chunks;
  a.out = L.out;
  a.ldo = L.ldo;
  a.err = L.err;
  auto kern = k_gemm_experts<kOutBF16>;
  static PerDevice attr_set = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_set[dev] = 1;
  }
  // At most one tile per expert that has rows, plus one per 256 rows, times the weight tiles.
  const long long most = ((long long)(L.E < L.T ? L.E : L.T) + L.T / kTileN) * a.tiles_m;
  const int pairs = sm_count() / 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)(most < pairs ? most : pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, tm_w, tm_sfw, tm_x8, tm_x32, a);
}

}  // namespace

cudaError_t launch_gemm_experts(const ExpertsLaunch& L, cudaStream_t stream) {
  return L.out_bf16 ? launch_impl<true>(L, stream) : launch_impl<false>(L, stream);
}

}  // namespace batq
