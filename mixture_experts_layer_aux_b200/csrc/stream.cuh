// stream.cuh -- the gated feed-forward block for few tokens (one token of a
// decoding step up to MAX_T), where the time is that of streaming the weights
// through the SMs once.
//
// The product is taken transposed on the tensor cores: the weights are the M
// side (128 rows of an MMA), the tokens the N side, so nothing is padded to 128
// tokens. What would be the tile's height is free instead: a CTA owns
// r = ceil(rows / SMs) weight rows (the height of its TMA boxes, any number up
// to 128), so that every SM streams the same number of bytes, and K is split over
// CTAs only where a cluster shares a tile (plan()), through shared memory.
//   gate/up  r columns of F: r rows of W_g and r rows of W_u; the SwiGLU (MXFP8:
//            and the 1x32 quantisation of the activation, r a multiple of 32)
//            is the epilogue;
//   down     r rows of W_d.
// Where r is small, an MMA of 128 rows would be mostly empty and, at about 45
// clocks whatever its N up to 16, set the pace instead of memory. So s blocks of
// K (128 bytes per row each) are stacked: rows c r + i of the operand are K block
// c of weight row i, rows c T + t of the other are block c of token t, and the
// accumulator's diagonal blocks (c, c), added in the epilogue, are the result.
// With 2 s r <= 128, W_u's rows follow W_g's in the same operand. The boxes are
// three-dimensional (128 bytes x rows x s blocks): one copy per operand and
// stage, since small copies cost as much as large ones (on B200 a stage of
// 3.5 + 2 KB took 240 ns, whatever was done with it).
// Operand rows that no box fills read whatever lies behind it in shared memory;
// a row (column) of the accumulator depends on its own operand row alone, and
// those are not stored.
// Where there is little to stream, the ring leaves room for a second CTA: the
// down kernel starts while the gate/up kernel ends (programmatic dependent
// launch), and its first weights, which depend on nothing, are on their way
// before it waits for the activation.
//
// Once the gate/up kernel's last weights are on their way, its producer asks
// for the down kernel's to be brought into L2, so that memory stays busy while
// the one ends and the other begins.
//
// Roles (384 threads): warp 0 TMA producer, warp 1 MMA issuer and TMEM owner,
// warp 2 loader of the MXFP8 scales (natural [rows, K/32] layout -> the chunk
// order of the tensor-memory copies, see gemm_mx.cuh), warps 4..11 epilogue
// (TMEM lane quadrant w % 4, every other 16 tokens). Every wait is bounded
// (MOE_WAIT_NS).
#pragma once

#include "common.cuh"
#include "elect.cuh"
#include "gemm_mx.cuh"
#include "swiglu.cuh"

namespace moe_host {
// 3-D tiled map {inner, rows, blocks} with byte strides of rows and blocks, 128-byte swizzle, zero fill.
bool encode_tmap_3d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t rows,
                    uint64_t blocks, uint64_t row_stride, uint64_t block_stride, uint32_t box_inner,
                    uint32_t box_rows, uint32_t box_blocks);
}  // namespace moe_host

namespace stream {

constexpr int MAX_T = 56, MAX_T_MX = 16;
constexpr int MAX_STAGES = 16;
constexpr int EPI_WARP0 = 4, EPI_WARPS = 8;
constexpr int NUM_THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
// Kernels whose tiles may be shared by a cluster.
constexpr bool clusters(bool mx, bool gateup) { return mx || !gateup; }
constexpr int ROW_BYTES = 128;            // K bytes of a stage row (64 bf16 or 128 e4m3)
constexpr int OPERAND_BYTES = 128 * ROW_BYTES;  // what an MMA reads of its weight operand, filled or not
constexpr int MAX_N = 224;                // s T at most (two accumulators and the scales in 512 TMEM columns)
// MXFP8: stages of scales in shared memory, and how many the loader asks for ahead of the one it hands over (8 tokens,
// H = 7168, F = 2048: 24.4 us with 1, 23.2 with 2, 24.4 with 4, 24.9 with 8, whose first stage is late). It has then
// waited for the operands' stage, so the slot of SF_SLOTS stages before is free where the ring has no more than
// SF_SLOTS - SF_AHEAD stages.
constexpr int SF_SLOTS = 8, SF_AHEAD = 2;
constexpr int SF_SLOT_COLS = 12;          // scale columns of a stage in TMEM (W0, W1, x: 128 rows each)
constexpr int MAX_BLOCKS = 8, MAX_BLOCKS_MX = 4;  // K blocks of a stage
constexpr int MAX_CLUSTER = 4;            // CTAs that share a tile, each taking a part of K
constexpr int BAR_BYTES = 1024;
// Bytes of the ring. A CTA with little to stream (up to SHORT_BYTES in all) leaves room for one of the other kernel
// on its SM, which then starts while it runs; with much to stream, bytes in flight count: about 2 us of latency at
// 46 GB/s per SM (T = 1, H = 4096, F = 14336 bf16, with an earlier form of these kernels: 65 us with the large rings, 70
// with the shared ones; MXFP8 H = 7168, F = 2048: 32.4 and 28.7).
constexpr int RING_GATEUP = 116 * 1024, RING_DOWN = 100 * 1024, RING_ALONE = 200 * 1024;
constexpr int SHORT_BYTES = 512 * 1024;
constexpr int SMEM_FIXED = 1024 + BAR_BYTES;

struct __align__(64) Params {
  CUtensorMap tmW0, tmW1, tmX;
  CUtensorMap tmW0t, tmW1t, tmXt;   // the part of K past its last whole block (tail != 0): 2-D maps
  CUtensorMap tmNext;               // gate/up: the down kernel's W0, its rows per tile, blocks per stage, tiles, CTAs
  int next_r, next_s, next_tiles;   // per tile and stages, and which stages of a CTA's part of K to bring into L2
  int next_cs, next_KS;             // (from, to)
  int next_from, next_to;
  const uint8_t *sf0, *sf1, *x_sf;  // MXFP8 scales, [rows, K/32]
  void* out;                        // gate/up: bf16 or e4m3 codes; down: bf16; rows of ldo elements
  long long ldo;
  uint8_t* out_sf;                  // MXFP8 gate/up: [T, N/32]
  uint16_t* save_hi;                // bf16 gate/up: pre-activations (swiglu.cuh), rows of ld2, up from column `up`; or
  uint8_t* save_lo;                 // NULL
  long long ld2;
  int up;
  int T, N, K;                      // tokens, weight rows, reduction length
  int r, s;                         // weight rows per tile, K blocks per stage
  int KB, KS;                       // K blocks (128 bytes), stages of s blocks
  int w_rows;                       // s r rounded up to 8: operand rows of one weight
  int mma_n;                        // s T rounded up to 16
  int z;                            // tensor maps are cut along K; else s = 1
  int tail;                         // K % 64 elements follow the whole blocks (bf16, one tile per CTA)
  int r8, tail_n;                   // r rounded up to 8, T to 16: operand rows of the tail
  int tail_bytes;                   // its place in shared memory, before the ring
  int tiles;
  int stages, stage_bytes;
  int ring_bytes;                   // the stages, and what the last one's operands read past it
  int sf_w1, sf_x, sf_bytes;        // MXFP8: offsets of W1's and x's chunks in a slot of scales, and its size
  int cs;                           // CTAs per tile (a cluster, each with a part of K; MXFP8 gate/up, down)
  int acc_cols, acc_bufs, tmem_cols;  // TMEM: columns of one accumulator set, sets, allocation
  int early;                        // launched over the tail of the kernel that makes x
  int merged;                       // gate/up: both weights in one operand
  int staged;                       // the epilogue goes through shared memory (s > 1, merged or cs > 1)
  int* status;
};


// Instruction descriptors: bf16 (common.cuh) and MXFP8 (gemm_mx.cuh) with a run-time N.
template <bool MX>
MOE_DEV uint32_t idesc(int N, int q) {
  return MX ? ggmx::idesc_mx(128, N, q) : idesc_bf16(128, N, 0, 0);
}

MOE_DEV void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// 3-D tile: x (elements), row, K block.
MOE_DEV void tma_load_3d(void* smem_dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

MOE_DEV void tma_prefetch_3d(const CUtensorMap* m, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

MOE_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same shared-memory address in CTA `rank` of the cluster, and a store there.
MOE_DEV uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
MOE_DEV void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// First stage of a tile's CTA `rank` of cs (1, 2 or 4), each of which takes a part of the KS stages.
__host__ __device__ inline int part_of_k(int rank, int KS, int cs) { return rank * KS >> (cs >> 1); }

// The stages of the down kernel's CTA j (tile j / cs, rank j % cs; cs is 1 or 2) to bring into L2: [from, to).
__host__ __device__ inline void next_stages(const Params& p, int j, int& from, int& to) {
  const int rank = j & (p.next_cs - 1), k0 = part_of_k(rank, p.next_KS, p.next_cs);
  const int k1 = part_of_k(rank + 1, p.next_KS, p.next_cs);
  from = k0 + p.next_from;
  to = k0 + p.next_to < k1 ? k0 + p.next_to : k1;
}

// 4-byte asynchronous copy global -> shared; bytes 0: the destination is zeroed, nothing is read.
MOE_DEV void cp_async4(void* smem_dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(smem_dst)), "l"(src), "r"(bytes)
               : "memory");
}
MOE_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups have landed.
template <int N>
MOE_DEV void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where an operand row's scale word lies in its chunks.
MOE_DEV int chunk_offset(int row) { return 512 * (row >> 7) + 16 * (row & 31) + 4 * ((row >> 5) & 3); }

// Quantises one element per lane of a 32-lane block (fp32 a; NaN does not enter the maximum, as fmaxf).
MOE_DEV uint8_t quant_lane(float a, uint8_t& sb) {
  const float am = fmaxf(fabsf(a), 0.f);
  sb = ggmx::mx_scale_byte(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(am))));
  return __nv_cvt_float_to_fp8(a * ggmx::mx_inv_scale(sb), __NV_SATFINITE, __NV_E4M3);
}

MOE_DEV void save_preact(const Params& p, int tok, int col, float g, float u) {
  const long long at = tok * p.ld2 + col;
  p.save_hi[at] = (uint16_t)(__float_as_uint(g) >> 16);
  p.save_lo[at] = (uint8_t)(__float_as_uint(g) >> 8);
  p.save_hi[at + p.up] = (uint16_t)(__float_as_uint(u) >> 16);
  p.save_lo[at + p.up] = (uint8_t)(__float_as_uint(u) >> 8);
}

template <bool MX, bool GATEUP>
__global__ void __launch_bounds__(NUM_THREADS, 2) gemm_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* tail = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = tail + p.tail_bytes;
  uint8_t* sf_ring = ring + p.ring_bytes;
  uint8_t* bar_area = sf_ring + (MX ? SF_SLOTS * p.sf_bytes : 0);
  uint64_t* full = reinterpret_cast<uint64_t*>(bar_area);
  uint64_t* empty = full + MAX_STAGES;
  uint64_t* tfull = empty + MAX_STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* tail_full = tempty + 2;
  uint64_t* drain = tail_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w_bytes = p.w_rows * ROW_BYTES;
  const int x_off = (GATEUP ? 2 : 1) * w_bytes;
  // cs consecutive CTAs (a cluster) share a tile; this one takes the stages [ks0, ks1) of K, the first the tail too
  constexpr bool CLUSTER = clusters(MX, GATEUP);
  const int rank = CLUSTER ? (int)blockIdx.x % p.cs : 0;
  const int tile0 = CLUSTER ? (int)blockIdx.x / p.cs : (int)blockIdx.x;
  const int tile_step = CLUSTER ? (int)gridDim.x / p.cs : (int)gridDim.x;
  const int ks0 = CLUSTER ? part_of_k(rank, p.KS, p.cs) : 0, ks1 = CLUSTER ? part_of_k(rank + 1, p.KS, p.cs) : p.KS;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], MX ? 2 : 1);  // the producer, and the loader of scales
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], EPI_WARPS);
    }
    mbar_init(tail_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 32 * 3) {
    tma_prefetch_desc(&p.tmW0);
    if (GATEUP) tma_prefetch_desc(&p.tmW1);
    tma_prefetch_desc(&p.tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch_dependents();

  const bool with_tail = !MX && p.tail && rank == 0;

  bool aborted = false;
  if (warp == 0) {
    // ======================= TMA producer
    const uint32_t tx = (uint32_t)(((GATEUP ? 2 : 1) * p.r + p.T) * p.s * ROW_BYTES);
    const int kstep = MX ? 128 : 64;
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_par = 0;
    // the ks-th stage of K: coordinate along K, or the block's number where the maps are cut along it
    const auto load = [&](const CUtensorMap* m, int row, int ks, uint8_t* dst, uint64_t* bar) {
      const int kb = ks * p.s;
      tma_load_3d(dst, m, p.z ? 0 : kb * kstep, row, p.z ? kb : 0, bar);
    };
    const auto load_w = [&](int t, int ks, int st) {
      uint8_t* b = ring + st * p.stage_bytes;
      mbar_arrive_expect_tx(&full[st], tx);
      load(&p.tmW0, t * p.r, ks, b, &full[st]);
      if (GATEUP) load(&p.tmW1, t * p.r, ks, b + w_bytes, &full[st]);
    };
    // the first weights, before the wait for the kernel that makes x (where there is none, a stage's tokens go out
    // with its weights: behind the whole ring's they would be late)
    const int ahead = p.early ? min(p.stages, ks1 - ks0) : 0;
    for (int st = 0; st < ahead; ++st) {
      issued_mask |= 1u << st;
      if (elect_one()) load_w(tile0, ks0 + st, st);
    }
    if (with_tail && elect_one()) {
      mbar_arrive_expect_tx(tail_full, (uint32_t)(((GATEUP ? 2 : 1) * p.r + p.T) * ROW_BYTES));
      tma_load_2d(tail, &p.tmW0t, p.KB * kstep, tile0 * p.r, tail_full);
      if (GATEUP) tma_load_2d(tail + p.r8 * ROW_BYTES, &p.tmW1t, p.KB * kstep, tile0 * p.r, tail_full);
    }
    __syncwarp();
    griddep_wait();
    if (with_tail && elect_one())
      tma_load_2d(tail + (GATEUP ? 2 : 1) * p.r8 * ROW_BYTES, &p.tmXt, p.KB * kstep, 0, tail_full);
    __syncwarp();
    for (int t = tile0; t < p.tiles && !aborted; t += tile_step) {
      for (int ks = ks0; ks < ks1; ++ks) {
        const bool early = t == tile0 && ks < ks0 + ahead;
        if (!early) {
          if (!mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, p.status, DEV_WAIT_TIMEOUT_PRODUCER)) {
            aborted = true;
            break;
          }
          issued_mask |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        }
        if (elect_one()) {
          if (!early) load_w(t, ks, stage);
          load(&p.tmX, 0, ks, ring + stage * p.stage_bytes + x_off, &full[stage]);
        }
        __syncwarp();
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (GATEUP && elect_one())
      for (int j = blockIdx.x; j < p.next_tiles * p.next_cs && !aborted; j += gridDim.x) {
        int ks, to;
        next_stages(p, j, ks, to);
        for (; ks < to; ++ks) tma_prefetch_3d(&p.tmNext, 0, (j >> (p.next_cs >> 1)) * p.next_r, ks * p.next_s);
      }
    __syncwarp();
    if (*abort_flag) {
      // every TMA issued here must land before the CTA exits (a stage whose tokens were not asked for any more never
      // completes: the wait is bounded)
      const uint64_t t0 = globaltimer_ns();
      for (int i = 0; i < p.stages; ++i)
        if (issued_mask & (1u << i)) {
          const uint32_t par = (issued_par >> i) & 1u;
          while (!mbar_try_wait(&full[i], par) && globaltimer_ns() - t0 < MOE_WAIT_NS) {
          }
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ======================= MMA issuer. Descriptors are those of the first stage plus the address / 16.
    const bool two = GATEUP && !p.merged;
    const uint64_t desc0 = smem_desc_sw128(smem_u32(ring), 16, 1024);
    const uint64_t sdesc0 = ggmx::sf_desc(smem_u32(sf_ring));
    const uint32_t stage16 = p.stage_bytes >> 4, w16 = w_bytes >> 4, x16 = x_off >> 4;
    const uint32_t sf_tmem = tmem_base + p.acc_bufs * p.acc_cols;
    uint32_t id[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) id[q] = idesc<MX>(p.mma_n, q);
    int stage = 0, slot = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    const auto step = [&] {
      if (MX && ++slot == SF_SLOTS) slot = 0;
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1;
      }
    };
    for (int t = tile0; t < p.tiles && !aborted; t += tile_step) {
      if (!mbar_wait_warp(&tempty[acc], acc_phase ^ 1, abort_flag, p.status, DEV_WAIT_TIMEOUT_MMA)) {
        aborted = true;
        break;
      }
      tc_fence_after();
      const uint32_t d0 = tmem_base + acc * p.acc_cols, d1 = d0 + p.mma_n;
      bool first = true, slot2 = false;
      for (int ks = ks0; ks < ks1; ++ks) {
        if (!mbar_wait_warp(&full[stage], phase, abort_flag, p.status, DEV_WAIT_TIMEOUT_MMA)) {
          aborted = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t ad = desc0 + stage * stage16, bd = ad + x16;
          // scale slots of TMEM alternate: the copies of a stage follow, in issue order, the MMAs that read the slot
          // two stages ago
          const uint32_t sc = sf_tmem + (slot2 ? SF_SLOT_COLS : 0);
          if (MX) {
            const uint64_t sd = sdesc0 + slot * (p.sf_bytes >> 4), sx = sd + (p.sf_x >> 4);
            ggmx::tmem_cp_32x128b_x4(sc, sd);
            if (two) ggmx::tmem_cp_32x128b_x4(sc + 4, sd + (512 >> 4));
            ggmx::tmem_cp_32x128b_x4(sc + 8, sx);
          }
          const auto mma = [&](uint32_t d, uint64_t a, uint32_t sa, int q) {
            const uint32_t on = !first || q != 0 ? 1u : 0u;
            if (MX)
              ggmx::mma_mxf8(d, a + 2 * q, bd + 2 * q, id[q], sa | ((uint32_t)q << 30), (sc + 8) | ((uint32_t)q << 30),
                             on);
            else
              mma_bf16(d, a + 2 * q, bd + 2 * q, id[q], on);
          };
          if (two) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              mma(d0, ad, sc, q);
              mma(d1, ad + w16, sc + 4, q);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) mma(d0, ad, sc, q);
          }
          mma_commit(&empty[stage]);
        }
        __syncwarp();
        slot2 = !slot2;
        first = false;
        step();
      }
      if (aborted) break;
      if (with_tail) {
        // into accumulators of its own: its operands' rows are not stacked
        if (!mbar_wait_warp(tail_full, 0, abort_flag, p.status, DEV_WAIT_TIMEOUT_MMA)) {
          aborted = true;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t at = smem_desc_sw128(smem_u32(tail), 16, 1024), wt = p.r8 * ROW_BYTES >> 4;
          const uint64_t bt = at + (GATEUP ? 2 : 1) * wt;
          const uint32_t dt = tmem_base + p.acc_bufs * p.acc_cols, idt = idesc<MX>(p.tail_n, 0);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            mma_bf16(dt, at + 2 * q, bt + 2 * q, idt, q != 0 ? 1u : 0u);
            if (two) mma_bf16(dt + p.tail_n, at + wt + 2 * q, bt + 2 * q, idt, q != 0 ? 1u : 0u);
          }
        }
        __syncwarp();
      }
      if (elect_one()) mma_commit(&tfull[acc]);
      __syncwarp();
      if (++acc == p.acc_bufs) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
    if (*abort_flag) {
      // wait for every MMA already issued before TMEM is released
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < MOE_WAIT_NS) {
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ======================= MXFP8 scales. A chunk holds 128 operand rows: row 32 i + l in bytes 16 l + 4 i .. + 3,
    // one byte per 1x32 block of a K block. Every word goes from its place in the natural layout to its place in the
    // chunk by a 4-byte asynchronous copy, SF_AHEAD stages before it is needed (through registers, with the next four
    // K blocks loaded ahead, the loads' latency set the pace). The scales then join the operands' stage: the loader
    // waits for it as the producer does, and arrives on its barrier.
    if constexpr (MX) {
      const int kw = p.K / 32;  // scale bytes per row
      // Lane l copies the words of operand rows l + 32 j: block c = row / r of weight row (token) row % r. A block
      // past the end of K (of a last stage) or a row past the weights is zero-filled.
      constexpr int WJ = 4, XJ = 4 * MAX_T_MX / 32;
      const uint8_t *w0[WJ], *xs[XJ];
      int wc[WJ], wb[WJ], wd[WJ], xc[XJ];
      const long long w1 = GATEUP ? p.sf1 - p.sf0 : 0;
      const auto rows = [&](int t) {
#pragma unroll
        for (int j = 0; j < WJ; ++j) {
          const int e = lane + 32 * j, c = (e >= p.r) + (e >= 2 * p.r) + (e >= 3 * p.r), i = e - c * p.r;  // s <= 4
          const long long n = (long long)t * p.r + i;
          const bool in = e < p.s * p.r && n < p.N;
          w0[j] = in ? p.sf0 + n * kw + 4 * c : p.sf0;
          wc[j] = in ? c : 1 << 20;
          wb[j] = in ? 4 : 0;
          wd[j] = p.merged ? chunk_offset(e + p.w_rows) : p.sf_w1 + chunk_offset(e);
        }
      };
      rows(tile0);
#pragma unroll
      for (int j = 0; j < XJ; ++j) {
        const int e = lane + 32 * j, c = (e >= p.T) + (e >= 2 * p.T) + (e >= 3 * p.T);
        xs[j] = p.x_sf + (long long)(e - c * p.T) * kw + 4 * c;
        xc[j] = c;
      }
      // (the loader's instructions set the pace of short stages: whole stages go without the checks of the last)
      const int wn = p.s * p.r, xn = p.s * p.T;
      const auto weights = [&](int ks, int st) {
        uint8_t* sf = sf_ring + st * p.sf_bytes;
        if ((ks + 1) * p.s <= p.KB) {
          const long long at = 4 * ks * p.s;
#pragma unroll
          for (int j = 0; j < WJ; ++j) {
            if (32 * j >= wn) break;
            if (lane + 32 * j < wn) {
              cp_async4(sf + 16 * lane + 4 * j, w0[j] + at, wb[j]);
              if (GATEUP) cp_async4(sf + wd[j], w0[j] + at + w1, wb[j]);
            }
          }
          return;
        }
#pragma unroll
        for (int j = 0; j < WJ; ++j) {
          if (lane + 32 * j >= p.s * p.r) continue;
          const bool ok = ks * p.s + wc[j] < p.KB;
          const uint8_t* src = ok ? w0[j] + 4 * ks * p.s : p.sf0;
          cp_async4(sf + 16 * lane + 4 * j, src, ok ? 4 : 0);
          if (GATEUP) cp_async4(sf + wd[j], ok ? src + w1 : p.sf1, ok ? 4 : 0);
        }
      };
      const auto tokens = [&](int ks, int st) {
        uint8_t* sf = sf_ring + st * p.sf_bytes + p.sf_x;
        if ((ks + 1) * p.s <= p.KB) {
          const long long at = 4 * ks * p.s;
#pragma unroll
          for (int j = 0; j < XJ; ++j) {
            if (32 * j >= xn) break;
            if (lane + 32 * j < xn) cp_async4(sf + 16 * lane + 4 * j, xs[j] + at, 4);
          }
          return;
        }
#pragma unroll
        for (int j = 0; j < XJ; ++j) {
          if (lane + 32 * j >= p.s * p.T) continue;
          const bool ok = ks * p.s + xc[j] < p.KB;
          cp_async4(sf + 16 * lane + 4 * j, ok ? xs[j] + 4 * ks * p.s : p.x_sf, ok ? 4 : 0);
        }
      };
      // The next item to ask for: stage iks of tile it, into slot islot.
      int it = tile0, iks = ks0, islot = 0;
      const auto advance = [&] {
        if (++islot == SF_SLOTS) islot = 0;
        if (++iks == ks1) {
          iks = ks0;
          it += tile_step;
          if (it < p.tiles) rows(it);
        }
      };
      const int ahead = min(SF_AHEAD, ks1 - ks0);  // the weights', before the wait for the tokens'
      for (int j = 0; j < ahead; ++j) weights(ks0 + j, j);
      griddep_wait();
      for (int j = 0; j < SF_AHEAD; ++j) {
        if (it < p.tiles) {
          if (j >= ahead) weights(iks, islot);
          tokens(iks, islot);
          advance();
        }
        cp_async_commit();
      }
      int stage = 0;
      uint32_t phase = 0;
      for (int t = tile0; t < p.tiles && !aborted; t += tile_step) {
        for (int ks = ks0; ks < ks1; ++ks) {
          if (!mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, p.status, DEV_WAIT_TIMEOUT_PRODUCER)) {
            aborted = true;
            break;
          }
          if (it < p.tiles) {
            weights(iks, islot);
            tokens(iks, islot);
            advance();
          }
          cp_async_commit();
          cp_async_wait<SF_AHEAD>();
          fence_proxy_async_smem();  // written by ordinary copies, read by tcgen05.cp
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[stage]);
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      cp_async_wait<0>();  // (after an abort) no copy outlives the CTA
    }
  } else if (warp >= EPI_WARP0) {
    // ======================= epilogue: TMEM lanes 32 q .. 32 q + 31 = rows of the tile, columns = tokens
    griddep_wait();  // what the kernel before this one still reads may be what is written here
    const int q = warp & 3, h = (warp - EPI_WARP0) >> 2;
    const int row = 32 * q + lane;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = tile0; t < p.tiles && !aborted; t += tile_step) {
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], acc_phase, abort_flag, p.status, DEV_WAIT_TIMEOUT_EPILOGUE))) {
        aborted = true;
        break;
      }
      tc_fence_after();
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + acc * p.acc_cols;
      const uint32_t tail_tb = tmem_base + ((uint32_t)(q * 32) << 16) + p.acc_bufs * p.acc_cols;
      const int n0 = t * p.r;
      const int rows = min(p.r, p.N - n0);
      if (p.staged) break;  // one tile per CTA, finished below
      const bool ok = row < rows;
      for (int c = 16 * h; c < p.T; c += 32) {
        float v[16], u[16], v2[16], u2[16];
        tmem_ld16(tb + c, v);
        if (GATEUP) tmem_ld16(tb + p.mma_n + c, u);
        tmem_ld_wait();
        if (with_tail) {
          tmem_ld16(tail_tb + c, v2);
          if (GATEUP) tmem_ld16(tail_tb + p.tail_n + c, u2);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] += v2[i];
            if (GATEUP) u[i] += u2[i];
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (c + i >= p.T) break;
          const long long o = (c + i) * p.ldo + n0 + row;
          if constexpr (GATEUP) {
            const float a = swiglu::act(v[i], u[i]);
            if (MX) {
              uint8_t sb;
              const uint8_t code = quant_lane(ok ? a : 0.f, sb);
              if (ok) {
                static_cast<uint8_t*>(p.out)[o] = code;
                if (lane == 0) p.out_sf[o >> 5] = sb;
              }
            } else if (ok) {
              static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(a);
              if (p.save_hi) save_preact(p, c + i, n0 + row, v[i], u[i]);
            }
          } else if (ok) {
            static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(v[i]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
      if (++acc == p.acc_bufs) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
  }
  if (p.staged) {
    // The parts of one element (the K blocks of a stage, the tail, the CTAs of a cluster) are on different lanes,
    // columns and SMs. The accumulators go to shared memory as they are (the ring, whose stages have all been read):
    // fp32 [CTA][operand][column][128 rows], column c T + t of block c, token t; then the tails', [operand][t][128].
    // The CTAs of a cluster divide the tokens: token t is finished by CTA t % cs, and the others write its columns
    // into that CTA's memory.
    const int cs = CLUSTER ? p.cs : 1, lc = cs >> 1;  // cs is 1, 2 or 4: its logarithm is cs / 2
    const int ops = GATEUP && !p.merged ? 2 : 1;
    const int Tl = (p.T + cs - 1) >> lc, cols = p.s * Tl;  // columns per CTA and operand, where they are finished
    float* const tails = reinterpret_cast<float*>(ring) + (size_t)cs * ops * cols * 128;
    __syncwarp();
    if (CLUSTER && cs > 1) cluster_sync();  // every CTA's ring is free
    if (warp >= EPI_WARP0) {
      tc_fence_after();
      const int q = warp & 3, h = (warp - EPI_WARP0) >> 2, row = 32 * q + lane;
      const uint32_t tq = tmem_base + ((uint32_t)(q * 32) << 16);
      // block c of K is in rows [c r, (c + 1) r) and columns [c T, (c + 1) T): the columns that this warp's rows need
      int e0 = 32 * q, e1 = e0 + 31;
      if (p.merged && e0 >= p.w_rows) {  // rows of W_u
        e0 -= p.w_rows;
        e1 -= p.w_rows;
      } else if (p.merged && e1 >= p.w_rows) {
        e0 = 0;
        e1 = p.w_rows;
      }
      const int j0 = min(e0 / p.r, p.s - 1) * p.T, j1 = (min(e1 / p.r, p.s - 1) + 1) * p.T;
      const int chunks = e0 < p.s * p.r ? (j1 - j0 + 15) >> 4 : 0;
      for (int i = h; i < ops * chunks; i += 2) {
        const int op = i >= chunks, j = j0 + 16 * (i - op * chunks);
        float v[16];
        tmem_ld16(tq + op * p.mma_n + j, v);
        tmem_ld_wait();
        if (!CLUSTER || cs == 1) {
          float* dst = reinterpret_cast<float*>(ring) + ((size_t)op * cols + j) * 128 + row;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (j + k < j1) dst[128 * k] = v[k];
        } else {
          int c = j / p.T, tok = j - c * p.T;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            if (j + k < j1) {
              const uint32_t at = ((uint32_t)((rank * ops + op) * cols + c * Tl + (tok >> lc)) * 128 + row) * 4;
              st_cluster(cluster_addr(smem_u32(ring), tok & (cs - 1)) + at, v[k]);
            }
            if (++tok == p.T) {
              tok = 0;
              ++c;
            }
          }
        }
      }
      for (int op = 0; op < ops; ++op) {
        if (with_tail) {
          for (int j = 16 * h; j < p.T; j += 32) {
            float v[16];
            tmem_ld16(tq + p.acc_cols + op * p.tail_n + j, v);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int tok = j + k;
              if (tok >= p.T) break;
              const uint32_t at = smem_u32(tails + (size_t)(op * Tl + (tok >> lc)) * 128 + row);
              st_cluster(cs > 1 ? cluster_addr(at, tok & (cs - 1)) : at, v[k]);
            }
          }
        }
      }
    }
    if (CLUSTER && cs > 1) cluster_sync();
    else __syncthreads();
    // a warp takes 32 columns of one token at a time, and adds the parts in the order of K
    const int n0 = tile0 * p.r, rows = min(p.r, p.N - n0);
    const int mine = (p.T - rank + cs - 1) >> lc;  // tokens of this CTA
    const int up = p.merged ? p.w_rows : cols * 128, up_tail = p.merged ? p.r8 : Tl * 128;
    for (int f0 = 0; f0 < rows; f0 += 32) {
      const int f = f0 + lane;
      const bool ok = f < rows;
      const float* st = reinterpret_cast<const float*>(ring) + (ok ? f : 0);
      for (int tl = warp; tl < mine; tl += NUM_THREADS / 32) {
        float g = 0.f, u = 0.f;
        for (int k = 0; k < cs; ++k) {
          const float* pt = st + ((size_t)k * ops * cols + tl) * 128;
          for (int c = 0; c < p.s; ++c, pt += Tl * 128 + p.r) {
            g += pt[0];
            if (GATEUP) u += pt[up];
          }
        }
        if (!MX && p.tail) {
          const float* pt = tails + (size_t)tl * 128 + (ok ? f : 0);
          g += pt[0];
          if (GATEUP) u += pt[up_tail];
        }
        const float a = GATEUP ? swiglu::act(g, u) : g;
        const int tok = (tl << lc) + rank;
        const long long o = tok * p.ldo + n0 + f;
        if (MX && GATEUP) {
          uint8_t sb;
          const uint8_t code = quant_lane(ok ? a : 0.f, sb);
          if (ok) {
            static_cast<uint8_t*>(p.out)[o] = code;
            if (lane == 0) p.out_sf[o >> 5] = sb;
          }
        } else if (ok) {
          static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(a);
          if (GATEUP && p.save_hi) save_preact(p, tok, n0 + f, g, u);
        }
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, p.tmem_cols);
  }
}

// Geometry of a launch: rows per tile, K blocks per stage, stages, accumulators. The tensor maps follow from it
// (boxes of 128 bytes x r rows, or T tokens, x s blocks).
template <bool MX, bool GATEUP>
Params plan(int T, int N, int K) {
  Params p{};
  p.T = T;
  p.N = N;
  p.K = K;
  const int kstep = MX ? 128 : 64;
  const int sms = moe_host::num_sms();
  // equal tiles of at most 128 rows, in as few rounds over the SMs as that allows; the MXFP8 activation's blocks
  // of 32 columns stay within a tile
  const int unit = MX && GATEUP ? 32 : 8;
  const auto cut = [&](int n) {  // over n CTAs or clusters
    const int rounds = (N + 128 * n - 1) / (128 * n);
    p.r = (N + rounds * n - 1) / (rounds * n);
    if (MX && GATEUP) p.r = (p.r + 31) / 32 * 32;
    if (p.r < unit) p.r = unit;
    p.tiles = (N + p.r - 1) / p.r;
  };
  cut(sms);
  p.cs = 1;
  // Every CTA reads all tokens' K range. Where that is more than the weights it streams, two share a tile of twice
  // the rows and half of K each (48 tokens, H = 4096, F = 14336: 202 MB of activations through L2 next to 117 MB of
  // down weights, halved).
  if (!GATEUP && p.tiles <= sms && 4 * T > 5 * p.r && K >= 32 * kstep) {
    p.cs = 2;
    cut(sms / 2);
  }
  p.r8 = (p.r + 7) / 8 * 8;
  const bool one = p.tiles * p.cs <= sms;  // one tile per CTA
  p.tail = one && K > kstep ? K % kstep : 0;
  p.tail_n = (T + 15) / 16 * 16;
  p.z = p.tail || K % kstep == 0;
  p.KB = p.z ? K / kstep : (K + kstep - 1) / kstep;
  // K blocks per stage, and gate and up in one operand or in two: what costs the MMA issuer least per block (measured
  // with one thread in its loop, in ns: a wait and a commit 150, an MMA 32 + N / 8, a copy of scales 60), as far as
  // operand rows, TMEM and the ring allow
  float best = 1e30f;
  for (int merged = 0; merged <= (GATEUP && one ? 1 : 0); ++merged)
    for (int s = 1; s <= (one && p.z ? (MX ? MAX_BLOCKS_MX : MAX_BLOCKS) : 1); s += MX ? s : 1) {
      const int rows = (s * p.r + 7) / 8 * 8, n = (s * T + 15) / 16 * 16, ops = GATEUP && !merged ? 2 : 1;
      if (rows * (merged ? 2 : 1) > 128 || (s > 1 && (s * T > MAX_N || s > p.KB))) continue;
      const int stage = (GATEUP ? 2 : 1) * rows * ROW_BYTES + n * ROW_BYTES;
      const int cols = ops * n + (MX ? 2 * SF_SLOT_COLS : 16) + (p.tail ? ops * p.tail_n : 0);
      if (s > 1 && (cols > 512 || 4 * stage > RING_ALONE - (MX ? SF_SLOTS * 1536 : 40 * 1024))) continue;
      // a staged epilogue's accumulators fit where the ring (four stages at least) was
      if ((s > 1 || merged) && 512 * ops * (s * (T + MAX_CLUSTER - 1) + (p.tail ? T + 1 : 0)) > 4 * stage) continue;
      const float cost = (150.f + 4 * ops * (32.f + n / 8.f) + (MX ? 60.f * (ops + 1) : 0.f)) / s;
      if (cost < best) {
        best = cost;
        p.s = s;
        p.merged = merged;
        p.w_rows = rows;
        p.mma_n = n;
      }
    }
  p.staged = p.merged || p.s > 1 || p.cs > 1;
  p.KS = (p.KB + p.s - 1) / p.s;
  p.tail_bytes = p.tail ? ((GATEUP ? 2 : 1) * p.r8 + p.tail_n) * ROW_BYTES : 0;
  if (MX && GATEUP && p.staged)
    while (2 * p.cs <= MAX_CLUSTER && 2 * p.cs * p.tiles <= sms && p.KS >= 8 * p.cs) p.cs *= 2;
  p.stage_bytes = (GATEUP ? 2 : 1) * p.w_rows * ROW_BYTES + p.mma_n * ROW_BYTES;
  p.sf_w1 = p.merged ? 0 : 512;
  p.sf_x = GATEUP && !p.merged ? 1024 : 512;
  p.sf_bytes = p.sf_x + 512;
  const int sf_ring = MX ? SF_SLOTS * p.sf_bytes : 0;
  const long long all = (long long)p.KS / p.cs * p.stage_bytes * ((p.tiles + sms - 1) / sms);
  const int used = sf_ring + p.tail_bytes;
  p.stages = ((GATEUP ? RING_GATEUP : RING_DOWN) - used) / p.stage_bytes;
  if (p.stages < 4 || all > SHORT_BYTES) p.stages = (RING_ALONE - used) / p.stage_bytes;
  p.stages = std::min(p.stages, MX ? SF_SLOTS - SF_AHEAD : MAX_STAGES);
  const int reach = (GATEUP && !p.merged ? p.w_rows * ROW_BYTES : 0) + OPERAND_BYTES;  // of the operands of a stage
  p.ring_bytes = p.stages * p.stage_bytes + (reach > p.stage_bytes ? reach - p.stage_bytes : 0);
  p.acc_cols = (GATEUP && !p.merged ? 2 : 1) * p.mma_n;
  // past the accumulators: the scales, or the tail's, or what a last read may pass them by
  const int more = MX ? 2 * SF_SLOT_COLS
                      : p.tail ? (GATEUP && !p.merged ? 2 : 1) * p.tail_n + 16 : p.s > 1 ? 16 : 0;
  p.acc_bufs = one || 2 * p.acc_cols + more > 512 ? 1 : 2;
  const int cols = p.acc_bufs * p.acc_cols + more;
  p.tmem_cols = 32;
  while (p.tmem_cols < cols) p.tmem_cols *= 2;
  p.status = moe_host::device_status_ptr();
  return p;
}

// Tensor map of a [rows, K] operand with rows of ld elements: boxes of 128 bytes x box rows x s blocks of K.
template <bool MX>
bool encode_map(CUtensorMap* m, const Params& p, const void* base, int rows, int box, long long ld) {
  const uint64_t eb = MX ? 1 : 2, step = MX ? 128 : 64;
  return moe_host::encode_tmap_3d(m, MX ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base,
                                  p.z ? step : (uint64_t)p.K, rows, p.z ? p.KB : 1, ld * eb, ROW_BYTES, step, box,
                                  p.s);
}

// The maps of one operand: the whole blocks, and the tail.
template <bool MX>
bool encode_maps(CUtensorMap* m, CUtensorMap* mt, const Params& p, const void* base, int rows, int box, long long ld) {
  if (!encode_map<MX>(m, p, base, rows, box, ld)) return false;
  return !p.tail || moe_host::encode_tmap_2d(mt, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, p.K, rows, (uint64_t)ld * 2,
                                             64, box);
}

// The weights [K, N] of the down product that follows a gate/up launch: up to NEXT_BYTES of them beyond what its
// CTAs' rings take, the same number of stages for each CTA, are asked into L2 (about what memory delivers while the one
// kernel ends and the other begins).
constexpr long long NEXT_BYTES = 48ll << 20;
template <bool MX>
bool plan_next(Params& p, const void* W_next) {
  const Params d = plan<MX, false>(p.T, p.K, p.N);
  if (!d.z) return true;  // small boxes of one block, not worth it
  p.next_r = d.r;
  p.next_s = d.s;
  p.next_tiles = d.tiles;
  p.next_cs = d.cs;
  p.next_KS = d.KS;
  p.next_from = d.stages;
  const long long n = d.stages + NEXT_BYTES / ((long long)d.tiles * d.cs * d.s * d.r * ROW_BYTES);
  p.next_to = (int)(n < d.KS ? n : d.KS);
  return encode_map<MX>(&p.tmNext, d, W_next, d.N, d.r, d.K);
}

// dep: the kernel before it in the stream is one of the same call's (the weights are not its results).
template <bool MX, bool GATEUP>
int launch(Params& p, cudaStream_t st, bool dep) {
  p.early = dep;
  auto kern = gemm_kernel<MX, GATEUP>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           RING_ALONE + OPERAND_BYTES + SMEM_FIXED) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  cudaLaunchConfig_t cfg{};
  const int sms = moe_host::num_sms();
  cfg.gridDim = dim3(p.cs > 1 ? p.tiles * p.cs : p.tiles < sms ? p.tiles : sms);
  cfg.blockDim = dim3(NUM_THREADS);
  cfg.dynamicSmemBytes = p.tail_bytes + p.ring_bytes + (MX ? SF_SLOTS * p.sf_bytes : 0) + SMEM_FIXED;
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  int n = 0;
  if (dep) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (p.cs > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = p.cs;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace stream
