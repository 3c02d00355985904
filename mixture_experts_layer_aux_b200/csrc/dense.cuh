// dense.cuh -- dense GEMMs of the gated feed-forward block on the sm_100a tensor
// cores (tcgen05 + TMEM + TMA), in bf16 for any M, and N, K multiples of 8:
//   gate/up   a   = silu(x W_g^T) * (x W_u^T)     (both projections in one tile: [gate | up] columns)
//   down      y   = a W_d^T
//   dgrad     dgu = SwiGLU backward of (dY W_d),  dX = dgate W_g + dup W_u
//   wgrad     dW  = dO^T act
// and the first two in MXFP8 (K % 128 == 0), with the scales of both operands
// copied to TMEM beside the accumulators.
// Everything past an edge of M, N or K is zero-filled by TMA on the way in and
// predicated on the way out, so no operand is padded.
//
// Four forms. Template CG:
//   1  a CTA computes 128 x BN (tcgen05 M128 K16);
//   2  a pair of CTAs on neighbouring SMs computes 256 x BN with cta_group::2:
//      each holds its 128 rows of A and half of B's, so every SM moves less
//      through L2 and shared memory per product.
// Template BN: 256, or 128 where that fills the SMs better. plan() chooses.
// Roles (320 threads, one CTA per SM, persistent), as in the grouped GEMM of
// gemm.cuh: warp 0 TMA producer, warp 1 MMA issuer (the pair's first CTA) and
// TMEM owner (two BN-column accumulators; one of 256 columns with MXFP8), warps
// 2..9 epilogue (lane quadrant w % 4, column half), with MXFP8 warp 10 loader of
// the scales. Every wait is bounded (MOE_WAIT_NS).
//
// Work split. Whole tiles go round robin over the CTAs (pairs) while they fill
// every SM. The tiles of a rest that would leave many idle for long are cut
// along K, into one piece per CTA (pair) where that can be, else as one line of
// k-blocks in equal pieces. Pieces leave fp32 partial accumulators in the
// workspace (at most two per CTA; a piece that holds a whole tile finishes it),
// and fixup_kernel adds them in the order of K and applies the epilogue, so
// results do not depend on timing.
//
// Times in the comments below compare variants within one run. The large cases
// are slower in long runs, under the power cap (8192 tokens in MXFP8, H = 7168,
// F = 2048: 265 us in runs of 2 ms, 308 in one of seconds; a training step of
// 4096 tokens, H = 4096, F = 14336: 2930 and 3400).
#pragma once

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "elect.cuh"
#include "gemm_mx.cuh"
#include "swiglu.cuh"

namespace dense {

constexpr int BM = 128, BK = 64, MAX_BN = 256;
constexpr int A_BYTES = BM * BK * 2;
constexpr int EPI_WARPS = 8;
constexpr int NUM_THREADS = 64 + 32 * EPI_WARPS;
constexpr int STG_ROW = 80;  // staging: 32 rows x (64 + 16) bytes per epilogue warp
constexpr int STG_BYTES = EPI_WARPS * 32 * STG_ROW;
constexpr int BAR_BYTES = 256;
constexpr int SF_KB = 4;  // MXFP8: k-blocks whose scales are read at once
constexpr int MAX_CTAS = 160;                            // CTAs of one launch (one per SM)
constexpr size_t SLOT_FLOATS = (size_t)BM * MAX_BN;          // one CTA's partial accumulator
constexpr size_t PART_BYTES = 2ull * MAX_CTAS * SLOT_FLOATS * sizeof(float);

enum Op : int {
  OP_GATEUP = 0,     // A = x, B = W_g | W_u rows (K-major): a, optionally gate/up
  OP_DOWN = 1,       // A, B K-major: bf16
  OP_DGRAD_ACT = 2,  // A = dY K-major, B = W_d MN-major: dgate | dup from the saved gate/up
  OP_DGRAD_X = 3,    // A = dgate then dup (K-major), B = W_g then W_u (MN-major): bf16
  OP_WGRAD = 4,      // A = dO^T, B = act^T (both MN-major): bf16; the second half's rows from A2 into C2
  OP_GATEUP_MX = 5,  // the first two in MXFP8: e4m3 operands with a scale per 1x32 block, the activation as such
  OP_DOWN_MX = 6,
};
constexpr bool is_mx(int op) { return op >= OP_GATEUP_MX; }
constexpr bool is_gateup(int op) { return op == OP_GATEUP || op == OP_GATEUP_MX; }

struct __align__(64) Params {
  CUtensorMap tmA, tmA2, tmB0, tmB1;
  int M, N;            // output rows (of one half) and columns
  int KB;              // k-blocks of 128 bytes
  int kb_split;        // OP_DGRAD_X: k-blocks of the first half
  int halves;          // OP_WGRAD: 2 for two stacked outputs of M rows each (A2, C2 the second), else 1
  int tiles_m, tiles_n;
  int tm_split;        // m-tiles of one half
  int n_fast, group;   // order of the tiles: n before m, and how many of the faster one before the slower moves on
  int n_full;          // tiles done whole, round robin
  int sk_tiles;        // tiles n_full .. n_full + sk_tiles - 1, cut along K
  int sk_per;          // k-blocks per CTA (pair) of those
  int sk_kb;           // length of a tile on their line, >= KB: a multiple of sk_per where pieces end with their tile
  float* part;
  __nv_bfloat16* C;
  __nv_bfloat16* C2;
  long long ldc;
  // Saved pre-activations (swiglu.cuh), written by OP_GATEUP (NULL: not kept) and read by OP_DGRAD_ACT, whose dgate |
  // dup have the same shape: rows of ld2 elements, up in columns `up` on
  __nv_bfloat16* save_hi;
  uint8_t* save_lo;
  long long ld2;
  int up;
  // MXFP8: scales [rows, ld_sf] of A and B, read 16 bytes at a time when sf16; OP_GATEUP_MX writes e4m3 to C and scales
  // [M, N / 32] to C_sf
  const uint8_t *sfa, *sfb0, *sfb1;
  long long ld_sf;
  int sf16;
  uint8_t* C_sf;
  int* status;
};

struct Seg {
  int tile;  // -1: no more
  int kb0, nkb;
  int slot;  // >= 0: partial accumulator to leave there
};

// The pieces of work of CTA (pair) w of n: first its cut of the k-block line, then whole tiles.
struct Walk {
  int w, u, end, t, step;
  MOE_DEV Walk(const Params& p, int w_, int n) {
    const int units = p.sk_tiles * p.sk_kb;
    w = w_;
    u = min(w * p.sk_per, units);
    end = min(u + p.sk_per, units);
    t = w;
    step = n;
  }
  MOE_DEV Seg next(const Params& p) {
    Seg s;
    if (u < end) {
      const int i = u / p.sk_kb;
      s.kb0 = u - i * p.sk_kb;  // < KB: no piece starts in the gap behind a tile
      s.nkb = min(p.KB - s.kb0, end - u);
      s.tile = p.n_full + i;
      s.slot = s.nkb == p.KB ? -1 : 2 * w + (s.kb0 > 0 ? 0 : 1);
      u = p.sk_kb > p.KB ? end : u + s.nkb;
      return s;
    }
    s.kb0 = 0;
    s.nkb = p.KB;
    s.slot = -1;
    s.tile = t < p.n_full ? t : -1;
    t += step;
    return s;
  }
};

template <int OP, int CG, int BN_>
struct Cfg {
  static constexpr int BN = BN_;
  static constexpr bool A_MN = OP == OP_WGRAD;
  static constexpr bool B_MN = OP >= OP_DGRAD_ACT && OP <= OP_WGRAD;
  static constexpr bool MX = is_mx(OP), GATEUP = is_gateup(OP);
  static constexpr int N_STEP = GATEUP ? BN / 2 : BN;           // output columns per tile
  static constexpr int B_ROWS = BN / CG;                        // of B, per CTA
  static constexpr int STAGE_BYTES = A_BYTES + B_ROWS * BK * 2;  // by TMA
  static constexpr int kStages = BN == 128 ? (CG == 2 ? 8 : 6) : CG == 2 ? 6 : 4;
  static constexpr int THREADS = NUM_THREADS + (MX ? 32 : 0);   // MXFP8: one warp for the scales
  static constexpr int SF_BLOCKS = (BM + BN) / 128;             // MXFP8: 512-byte scale chunks of a k-block
  static constexpr int SF_BYTES = MX ? SF_BLOCKS * 512 : 0;
  static constexpr int SMEM_BYTES = 1024 + kStages * (STAGE_BYTES + SF_BYTES) + STG_BYTES + BAR_BYTES;
  static constexpr int B_BOX = GATEUP ? BN / 2 : B_ROWS < 128 ? B_ROWS : 128;  // rows of a K-major B box
  // TMEM: accumulators, then two slots of scales (4 columns per chunk)
  static constexpr int ACCS = MX && BN == 256 ? 1 : 2;
  static constexpr int TMEM_COLS = MX ? 512 : 2 * BN;
  static_assert(!MX || ACCS * BN + 8 * SF_BLOCKS <= 512, "TMEM");
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

struct Origin {
  int m0, n0, rows, cols;  // m0, n0 within the (half) output, m0 of this CTA; rows, cols: valid extent (may be <= 0)
  bool second;             // OP_WGRAD: the second half
};
// rank: the CTA's place in its pair.
template <int OP, int CG, int BN>
MOE_DEV Origin origin(const Params& p, int tile, int rank) {
  Origin o;
  // the tiles of p.group rows (or columns) by turns, along all columns (rows)
  const int fast = p.n_fast ? p.tiles_n : p.tiles_m, slow = p.n_fast ? p.tiles_m : p.tiles_n;
  int f0 = 0, i = tile, w = fast;
  if (p.group < fast) {
    f0 = tile / (p.group * slow) * p.group;
    i -= f0 * slow;
    w = min(p.group, fast - f0);
  }
  const int st = i / w, ft = f0 + i - st * w;
  const int mt = p.n_fast ? st : ft, nt = p.n_fast ? ft : st;
  o.second = OP == OP_WGRAD && mt >= p.tm_split;
  o.m0 = (mt - (o.second ? p.tm_split : 0)) * BM * CG + rank * BM;
  o.n0 = nt * Cfg<OP, CG, BN>::N_STEP;
  o.rows = min(BM, p.M - o.m0);
  o.cols = min(Cfg<OP, CG, BN>::N_STEP, p.N - o.n0);
  return o;
}

// ---------------------------------------------------------------- CTA pairs

// Shared-memory address of the pair's CTA `rank`.
MOE_DEV uint32_t pair_addr(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
MOE_DEV void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <int CG>
MOE_DEV void load_tile(void* dst, const CUtensorMap* m, int x, int y, uint64_t* bar) {
  if constexpr (CG == 1) {
    tma_load_2d(dst, m, x, y, bar);
  } else {
    // the bytes are counted on the first CTA's barrier
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(pair_addr(smem_u32(bar), 0))
        : "memory");
  }
}
template <int CG>
MOE_DEV void mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 1)
    mma_bf16(d_tmem, adesc, bdesc, idesc, accumulate);
  else
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
template <int CG>
MOE_DEV void mma_mx(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                    uint32_t accumulate) {
  if constexpr (CG == 1)
    ggmx::mma_mxf8(d_tmem, adesc, bdesc, idesc, sfa, sfb, accumulate);
  else
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p; }" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}
// One chunk of scales (128 rows x 4 bytes) to 4 columns of TMEM; a pair: of both CTAs, each from its own.
template <int CG>
MOE_DEV void copy_sf(uint32_t taddr, uint64_t sdesc) {
  if constexpr (CG == 1)
    ggmx::tmem_cp_32x128b_x4(taddr, sdesc);
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
// Arrives on the barrier (of both CTAs of a pair) once every MMA issued so far is done.
template <int CG>
MOE_DEV void commit(uint64_t* bar) {
  if constexpr (CG == 1) {
    mma_commit(bar);
  } else {
#pragma unroll
    for (uint32_t r = 0; r < 2; ++r)
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                       pair_addr(smem_u32(bar), r))
                   : "memory");
  }
}
// Arrives on the first CTA's barrier, relaxed. For accumulators that is all: they are in registers (tcgen05.wait::ld
// and the tcgen05 fences order them). Scales are ordinary stores to this SM's shared memory which the first CTA's
// tcgen05.cp reads, and a proxy fence orders no threads: release_smem_cluster() goes before their arrival, and the
// issuer waits with the matching acquire. A release of all memory at the cluster's scope would also wait for every
// access to global memory in flight: 1 us per tile, and 0.9 us per k-block of MXFP8, whose MMAs take 0.35.
template <int CG>
MOE_DEV void arrive_first(uint64_t* bar) {
  if constexpr (CG == 1)
    mbar_arrive(bar);
  else
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(pair_addr(smem_u32(bar), 0))
                 : "memory");
}
template <int CG>
MOE_DEV void alloc_tmem(uint32_t* slot, uint32_t cols) {
  if constexpr (CG == 1) {
    tmem_alloc(slot, cols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
MOE_DEV void free_tmem(uint32_t taddr, uint32_t cols) {
  if constexpr (CG == 1)
    tmem_dealloc(taddr, cols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}

// 32 bf16 of each of the warp's 32 rows (16 words per lane, lane = row) to dst (row-contiguous through the
// warp's staging buffer: 4 lanes x 16 bytes per row). rows, cols: how many of the 32 x 32 exist (cols % 8 == 0).
MOE_DEV void store_rows(uint8_t* stg, const uint32_t (&w)[16], __nv_bfloat16* dst, long long ld, int rows, int cols) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(stg + lane * STG_ROW + 16 * j) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  __syncwarp();
  const int piece = lane & 3, r0 = lane >> 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + r0;
    if (r < rows && 8 * piece < cols)
      *reinterpret_cast<uint4*>(dst + r * ld + 8 * piece) =
          *reinterpret_cast<const uint4*>(stg + r * STG_ROW + 16 * piece);
  }
  __syncwarp();
}

// The reverse: 32 bf16 of each of the warp's rows into 16 words per lane (zero where they do not exist).
MOE_DEV void load_rows(uint8_t* stg, uint32_t (&w)[16], const __nv_bfloat16* src, long long ld, int rows, int cols) {
  const int lane = threadIdx.x & 31;
  const int piece = lane & 3, r0 = lane >> 2;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + r0;
    v[i] = make_uint4(0, 0, 0, 0);
    if (r < rows && 8 * piece < cols) v[i] = *reinterpret_cast<const uint4*>(src + r * ld + 8 * piece);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(stg + (8 * i + r0) * STG_ROW + 16 * piece) = v[i];
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 u = *reinterpret_cast<const uint4*>(stg + lane * STG_ROW + 16 * j);
    w[4 * j] = u.x;
    w[4 * j + 1] = u.y;
    w[4 * j + 2] = u.z;
    w[4 * j + 3] = u.w;
  }
  __syncwarp();
}

// The same for 32 bytes of each row (8 words per lane, 4 lanes x 8 bytes per row).
MOE_DEV void store_rows8(uint8_t* stg, const uint32_t (&w)[8], uint8_t* dst, long long ld, int rows, int cols) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    *reinterpret_cast<uint4*>(stg + lane * STG_ROW + 16 * j) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  __syncwarp();
  const int piece = lane & 3, r0 = lane >> 2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + r0;
    if (r < rows && 8 * piece < cols)
      *reinterpret_cast<uint2*>(dst + r * ld + 8 * piece) = *reinterpret_cast<const uint2*>(stg + r * STG_ROW + 8 * piece);
  }
  __syncwarp();
}
MOE_DEV void load_rows8(uint8_t* stg, uint32_t (&w)[8], const uint8_t* src, long long ld, int rows, int cols) {
  const int lane = threadIdx.x & 31;
  const int piece = lane & 3, r0 = lane >> 2;
  uint2 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + r0;
    v[i] = make_uint2(0, 0);
    if (r < rows && 8 * piece < cols) v[i] = *reinterpret_cast<const uint2*>(src + r * ld + 8 * piece);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) *reinterpret_cast<uint2*>(stg + (8 * i + r0) * STG_ROW + 8 * piece) = v[i];
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint4 u = *reinterpret_cast<const uint4*>(stg + lane * STG_ROW + 16 * j);
    w[4 * j] = u.x;
    w[4 * j + 1] = u.y;
    w[4 * j + 2] = u.z;
    w[4 * j + 3] = u.w;
  }
  __syncwarp();
}
MOE_DEV void split32(const float (&v)[32], uint32_t (&hi)[16], uint32_t (&lo)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[2 * i] = swiglu::hi2(v[4 * i], v[4 * i + 1]);
    hi[2 * i + 1] = swiglu::hi2(v[4 * i + 2], v[4 * i + 3]);
    lo[i] = swiglu::lo4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}

MOE_DEV void pack32(const float (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
}

template <int OP, int CG, int BN>
__global__ void __launch_bounds__(Cfg<OP, CG, BN>::THREADS, 1) gemm_kernel(const __grid_constant__ Params p) {
  using C = Cfg<OP, CG, BN>;
  constexpr int kStages = C::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sf_ring = smem + kStages * C::STAGE_BYTES;
  uint8_t* stg_area = sf_ring + kStages * C::SF_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg_area + STG_BYTES);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 2 ? (int)blockIdx.x & 1 : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], C::MX ? 1 + CG : 1);  // the producer, and the loaders of scales
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], CG * EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x == 64) {
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB0);
  }
  if (warp == 1) alloc_tmem<CG>(tmem_slot, C::TMEM_COLS);
  __syncthreads();
  if (CG == 2) pair_sync();  // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // launched over the tail of the kernel before it: its results are visible from here on
  griddep_wait();
  griddep_launch_dependents();

  bool aborted = false;
  Walk walk(p, (int)blockIdx.x / CG, (int)gridDim.x / CG);
  if (warp == 0) {
    // ======================= TMA producer: this CTA's rows of A and B
    int stage = 0;
    uint32_t phase = 0, issued_mask = 0, issued_par = 0;
    for (Seg s = walk.next(p); s.tile >= 0 && !aborted; s = walk.next(p)) {
      const Origin o = origin<OP, CG, BN>(p, s.tile, rank);
      const int b0 = o.n0 + (C::GATEUP ? 0 : rank * C::B_ROWS);
      for (int kb = s.kb0; kb < s.kb0 + s.nkb; ++kb) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, p.status, DEV_WAIT_TIMEOUT_PRODUCER)) {
          aborted = true;
          break;
        }
        issued_mask |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[stage], CG * C::STAGE_BYTES);
          uint8_t* sA = smem + stage * C::STAGE_BYTES;
          uint8_t* sB = sA + A_BYTES;
          uint64_t* bar = &full[stage];
          const bool hi = OP == OP_DGRAD_X && kb >= p.kb_split;  // the up half of K
          const int kc = (kb - (hi ? p.kb_split : 0)) * (C::MX ? 128 : BK);
          const CUtensorMap* mA = (hi || o.second) ? &p.tmA2 : &p.tmA;
          if constexpr (!C::A_MN) {
            load_tile<CG>(sA, mA, kc, o.m0, bar);
          } else {
            load_tile<CG>(sA, mA, o.m0, kc, bar);
            load_tile<CG>(sA + 64 * BK * 2, mA, o.m0 + 64, kc, bar);
          }
          if constexpr (C::GATEUP) {
            // the first half of the accumulator's columns is gate, the second up
            if constexpr (CG == 2) {
              load_tile<CG>(sB, rank ? &p.tmB1 : &p.tmB0, kc, b0, bar);
            } else {
              load_tile<CG>(sB, &p.tmB0, kc, b0, bar);
              load_tile<CG>(sB + BN / 2 * BK * 2, &p.tmB1, kc, b0, bar);
            }
          } else if constexpr (!C::B_MN) {
#pragma unroll
            for (int j = 0; j < C::B_ROWS / C::B_BOX; ++j)
              load_tile<CG>(sB + j * C::B_BOX * BK * 2, &p.tmB0, kc, b0 + C::B_BOX * j, bar);
          } else {
            const CUtensorMap* mB = hi ? &p.tmB1 : &p.tmB0;
#pragma unroll
            for (int j = 0; j < C::B_ROWS / 64; ++j) load_tile<CG>(sB + j * 64 * BK * 2, mB, b0 + 64 * j, kc, bar);
          }
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (CG == 2) {
      // no commit of the first CTA may arrive here after this CTA has left: wait until every stage is released
      for (int i = 0; i < kStages && !aborted; ++i) {
        if (!mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, p.status, DEV_WAIT_TIMEOUT_PRODUCER)) aborted = true;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (*abort_flag) {
      // every TMA issued here must land before the CTA exits (a pair's second CTA cannot see its own land: it gives
      // them a time)
      const uint64_t t1 = globaltimer_ns();
      for (int i = 0; i < kStages; ++i)
        if (issued_mask & (1u << i)) {
          const uint32_t par = (issued_par >> i) & 1u;
          while (rank == 0 && !mbar_try_wait(&full[i], par) && globaltimer_ns() - t1 < MOE_WAIT_NS) {
          }
        }
      while (CG == 2 && globaltimer_ns() - t1 < 1000000ull) {
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ======================= MMA issuer. Descriptors are those of the first stage plus the address / 16.
    if (rank == 0) {
      constexpr uint32_t IDESC = idesc_bf16(CG * BM, BN, C::A_MN ? 1 : 0, C::B_MN ? 1 : 0);
      const uint64_t sd0 = C::MX ? ggmx::sf_desc(smem_u32(sf_ring)) : 0;
      const uint32_t sf_tmem = tmem_base + C::ACCS * BN;
      int slot = 0;
      constexpr int A_STEP = (C::A_MN ? 2048 : 32) >> 4, B_STEP = (C::B_MN ? 2048 : 32) >> 4;  // 16 of K
      const uint32_t base = smem_u32(smem);
      const uint64_t a0 = smem_desc_sw128(base, C::A_MN ? 64 * BK * 2 : 16, 1024);
      const uint64_t b0 = smem_desc_sw128(base + A_BYTES, C::B_MN ? 64 * BK * 2 : 16, 1024);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      for (Seg s = walk.next(p); s.tile >= 0 && !aborted; s = walk.next(p)) {
        if (!mbar_wait_warp(&tempty[acc], acc_phase ^ 1, abort_flag, p.status, DEV_WAIT_TIMEOUT_MMA)) {
          aborted = true;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = 0; kb < s.nkb; ++kb) {
          bool ready;
          if constexpr (C::MX && CG == 2)  // the other CTA's scales too
            ready = mbar_wait_warp_cluster(&full[stage], phase, abort_flag, p.status, DEV_WAIT_TIMEOUT_MMA);
          else
            ready = mbar_wait_warp(&full[stage], phase, abort_flag, p.status, DEV_WAIT_TIMEOUT_MMA);
          if (!ready) {
            aborted = true;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t ad = a0 + stage * (C::STAGE_BYTES >> 4), bd = b0 + stage * (C::STAGE_BYTES >> 4);
            if constexpr (C::MX) {
              // slots alternate: the copies into one follow, in issue order, the MMAs that read it two k-blocks ago
              const uint32_t sc = sf_tmem + slot * 4 * C::SF_BLOCKS;
              const uint64_t sd = sd0 + stage * (C::SF_BYTES >> 4);
#pragma unroll
              for (int i = 0; i < C::SF_BLOCKS; ++i) copy_sf<CG>(sc + 4 * i, sd + i * (512 >> 4));
#pragma unroll
              for (int q = 0; q < 4; ++q)
                mma_mx<CG>(d_tmem, ad + 2 * q, bd + 2 * q, ggmx::idesc_mx(CG * BM, BN, q), sc | ((uint32_t)q << 30),
                           (sc + 4) | ((uint32_t)q << 30), (kb | q) != 0 ? 1u : 0u);
            } else {
#pragma unroll
              for (int kk = 0; kk < BK / 16; ++kk)
                mma<CG>(d_tmem, ad + kk * A_STEP, bd + kk * B_STEP, IDESC, (kb | kk) != 0 ? 1u : 0u);
            }
            commit<CG>(&empty[stage]);
          }
          __syncwarp();
          slot ^= 1;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (aborted) break;
        if (elect_one()) commit<CG>(&tfull[acc]);
        __syncwarp();
        if (++acc == C::ACCS) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      if (*abort_flag) {
        // wait for every MMA already issued before TMEM is released
        if (elect_one()) commit<CG>(drain);
        __syncwarp();
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < MOE_WAIT_NS) {
        }
      }
    }
    __syncwarp();
  } else if (C::MX && warp == 10) {
    // ======================= MXFP8 scales, of A's rows of this CTA and of all of B's of the tile (a pair: each CTA
    // needs all). They join their stage: the loader waits for the stage as the producer does, and arrives on its
    // barrier. A lane reads the words of SF_KB k-blocks of rows l, l + 32, l + 64, l + 96 of a block of 128, one batch
    // ahead, and writes, per k-block, these rows' words as the 16 bytes l of its chunk; one proxy fence for two
    // k-blocks, and no more instructions than that takes: they set the pace (8192 tokens, H = 7168, F = 2048, in short
    // runs: 270 us when it was made; with the rows' addresses computed for each batch 290, with a second loader and a
    // fence for each k-block besides 298, with barriers of their own for four k-blocks at a time 360).
    if constexpr (C::MX) {
      uint32_t cur[C::SF_BLOCKS][4][SF_KB], nxt[C::SF_BLOCKS][4][SF_KB];
      Seg s = walk.next(p);
      int base = s.kb0 / SF_KB * SF_KB;  // the batch in nxt: k-blocks base .. base + SF_KB - 1 of s
      const uint8_t* src[C::SF_BLOCKS][4];  // this lane's rows
      uint32_t in = 0;                       // which of them exist
      const auto rows = [&] {
        const Origin o = origin<OP, CG, BN>(p, s.tile, rank);
        in = 0;
#pragma unroll
        for (int b = 0; b < C::SF_BLOCKS; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 128 * b + 32 * i + lane, n = r - BM, c = C::GATEUP ? n % (BN / 2) : n;
            const bool ok = b == 0 ? r < o.rows : c < o.cols;
            if (b == 0) src[b][i] = p.sfa + (o.m0 + r) * p.ld_sf;
            else src[b][i] = (C::GATEUP && n >= BN / 2 ? p.sfb1 : p.sfb0) + (long long)(o.n0 + c) * p.ld_sf;
            in |= (ok ? 1u : 0u) << (4 * b + i);
          }
      };
      const auto fetch = [&] {
#pragma unroll
        for (int b = 0; b < C::SF_BLOCKS; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool ok = (in >> (4 * b + i)) & 1u;
            if (p.sf16) {
              const uint4 w = ok ? *reinterpret_cast<const uint4*>(src[b][i] + 4 * base) : make_uint4(0, 0, 0, 0);
              nxt[b][i][0] = w.x;
              nxt[b][i][1] = w.y;
              nxt[b][i][2] = w.z;
              nxt[b][i][3] = w.w;
            } else {
#pragma unroll
              for (int k = 0; k < SF_KB; ++k)
                nxt[b][i][k] = ok && base + k < p.KB ? reinterpret_cast<const uint32_t*>(src[b][i])[base + k] : 0;
            }
          }
      };
      int stage = 0;
      uint32_t phase = 0;
      if (s.tile >= 0) {
        rows();
        fetch();
      }
      while (s.tile >= 0 && !aborted) {
        const int k0 = max(s.kb0 - base, 0), k1 = min(s.kb0 + s.nkb - base, SF_KB);  // the batch's k-blocks
#pragma unroll
        for (int b = 0; b < C::SF_BLOCKS; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < SF_KB; ++k) cur[b][i][k] = nxt[b][i][k];
        base += SF_KB;
        if (base >= s.kb0 + s.nkb) {
          s = walk.next(p);
          base = s.kb0 / SF_KB * SF_KB;
          if (s.tile >= 0) rows();
        }
        if (s.tile >= 0) fetch();
#pragma unroll
        for (int k = 0; k < SF_KB; k += 2) {
          int st[2] = {-1, -1};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (k + j < k0 || k + j >= k1 || aborted) continue;
            if (!mbar_wait_warp(&empty[stage], phase ^ 1, abort_flag, p.status, DEV_WAIT_TIMEOUT_PRODUCER)) {
              aborted = true;
              continue;
            }
            uint8_t* dst = sf_ring + stage * C::SF_BYTES + 16 * lane;
#pragma unroll
            for (int b = 0; b < C::SF_BLOCKS; ++b)
              *reinterpret_cast<uint4*>(dst + b * 512) =
                  make_uint4(cur[b][0][k + j], cur[b][1][k + j], cur[b][2][k + j], cur[b][3][k + j]);
            st[j] = stage;
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (CG == 2) release_smem_cluster();
            if (st[0] >= 0) arrive_first<CG>(&full[st[0]]);
            if (st[1] >= 0) arrive_first<CG>(&full[st[1]]);
          }
        }
      }
    }
  } else {
    // ======================= epilogue: lane quadrant q, column half h
    const int ew = warp - 2, q = warp & 3, h = ew >> 2;
    uint8_t* stg = stg_area + ew * 32 * STG_ROW;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (Seg s = walk.next(p); s.tile >= 0 && !aborted; s = walk.next(p)) {
      if (!__all_sync(0xffffffffu, mbar_wait(&tfull[acc], acc_phase, abort_flag, p.status, DEV_WAIT_TIMEOUT_EPILOGUE))) {
        aborted = true;
        break;
      }
      tc_fence_after();
      const Origin o = origin<OP, CG, BN>(p, s.tile, rank);
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + acc * BN;
      bool released = false;
      const int rows = o.rows - 32 * q;  // of this warp's 32 (may be <= 0)
      const long long row0 = (long long)o.m0 + 32 * q;
      if (s.slot >= 0) {
        // fp32 partial, column-major: a warp store writes one column's 32 rows
        float* dst = p.part + (size_t)(s.slot * CG + rank) * SLOT_FLOATS + 32 * q + lane;
        const bool ok = lane < rows;
#pragma unroll 1
        for (int c = h * (BN / 2); c < (h + 1) * (BN / 2); c += 32) {
          float v[32];
          tmem_ld32(tb + c, v);
          tmem_ld_wait();
          if (ok)
#pragma unroll
            for (int i = 0; i < 32; ++i) dst[(size_t)(c + i) * BM] = v[i];
        }
      } else if constexpr (OP == OP_GATEUP) {
#pragma unroll 1
        for (int c = h * (BN / 4); c < (h + 1) * (BN / 4); c += 32) {
          const int cols = o.cols - c;
          if (cols <= 0) break;  // warp-uniform
          float g[32], u[32];
          uint32_t w[16];
          tmem_ld32(tb + c, g);
          tmem_ld32(tb + BN / 2 + c, u);
          tmem_ld_wait();
          if (p.save_hi) {
            const long long at = row0 * p.ld2 + o.n0 + c;
            uint32_t lo[8];
            split32(g, w, lo);
            store_rows(stg, w, p.save_hi + at, p.ld2, rows, cols);
            store_rows8(stg, lo, p.save_lo + at, p.ld2, rows, cols);
            split32(u, w, lo);
            store_rows(stg, w, p.save_hi + at + p.up, p.ld2, rows, cols);
            store_rows8(stg, lo, p.save_lo + at + p.up, p.ld2, rows, cols);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] = swiglu::act(g[i], u[i]);
          pack32(g, w);
          store_rows(stg, w, p.C + row0 * p.ldc + o.n0 + c, p.ldc, rows, cols);
        }
      } else if constexpr (C::MX) {
        // one accumulator (BN = 256): released as soon as its columns are in registers, so the next tile's MMAs run
        // beside what follows
        constexpr int NB = BN / 64;  // blocks of 32 columns of this warp: gate then up
        float v[NB][32];
#pragma unroll
        for (int j = 0; j < NB; ++j)
          tmem_ld32(tb + (C::GATEUP ? h * (BN / 4) + (j < NB / 2 ? 32 * j : BN / 2 + 32 * (j - NB / 2))
                                    : h * (BN / 2) + 32 * j),
                    v[j]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first<CG>(&tempty[acc]);
        released = true;
        if constexpr (C::GATEUP) {
#pragma unroll
          for (int j = 0; j < NB / 2; ++j) {
            const int c = h * (BN / 4) + 32 * j, cols = o.cols - c;
            float am = 0.f;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              v[j][i] = swiglu::act(v[j][i], v[j + NB / 2][i]);
              am = fmaxf(am, fabsf(v[j][i]));
            }
            const uint8_t sb = ggmx::mx_scale_byte(am);
            uint32_t w[8];
            ggmx::quant32(v[j], ggmx::mx_inv_scale(sb), w);
            store_rows8(stg, w, reinterpret_cast<uint8_t*>(p.C) + row0 * p.ldc + o.n0 + c, p.ldc, rows, cols);
            if (lane < rows && cols > 0) p.C_sf[((row0 + lane) * p.ldc + o.n0 + c) >> 5] = sb;
          }
        } else {
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const int c = h * (BN / 2) + 32 * j;
            uint32_t w[16];
            pack32(v[j], w);
            store_rows(stg, w, p.C + row0 * p.ldc + o.n0 + c, p.ldc, rows, o.cols - c);
          }
        }
      } else if constexpr (OP == OP_DGRAD_ACT) {
#pragma unroll 1
        for (int c = h * (BN / 2); c < (h + 1) * (BN / 2); c += 32) {
          const int cols = o.cols - c;
          if (cols <= 0) break;
          float v[32];
          uint32_t zg[16], zu[16], lg[8], lu[8];
          const long long at = row0 * p.ld2 + o.n0 + c;
          load_rows(stg, zg, p.save_hi + at, p.ld2, rows, cols);
          load_rows8(stg, lg, p.save_lo + at, p.ld2, rows, cols);
          load_rows(stg, zu, p.save_hi + at + p.up, p.ld2, rows, cols);
          load_rows8(stg, lu, p.save_lo + at + p.up, p.ld2, rows, cols);
          tmem_ld32(tb + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float g[4], u[4];
            swiglu::join4(zg[2 * i], zg[2 * i + 1], lg[i], g);
            swiglu::join4(zu[2 * i], zu[2 * i + 1], lu[i], u);
#pragma unroll
            for (int j = 0; j < 4; ++j) swiglu::grad(v[4 * i + j], g[j], u[j], g[j], u[j]);
            zg[2 * i] = pack_bf16x2(g[0], g[1]);
            zg[2 * i + 1] = pack_bf16x2(g[2], g[3]);
            zu[2 * i] = pack_bf16x2(u[0], u[1]);
            zu[2 * i + 1] = pack_bf16x2(u[2], u[3]);
          }
          store_rows(stg, zg, p.C + at, p.ld2, rows, cols);
          store_rows(stg, zu, p.C + at + p.up, p.ld2, rows, cols);
        }
      } else {
        __nv_bfloat16* base = (o.second ? p.C2 : p.C) + row0 * p.ldc + o.n0;
#pragma unroll 1
        for (int c = h * (BN / 2); c < (h + 1) * (BN / 2); c += 32) {
          const int cols = o.cols - c;
          if (cols <= 0) break;
          float v[32];
          uint32_t w[16];
          tmem_ld32(tb + c, v);
          tmem_ld_wait();
          pack32(v, w);
          store_rows(stg, w, base + c, p.ldc, rows, cols);
        }
      }
      if (!released) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first<CG>(&tempty[acc]);
      }
      if (++acc == C::ACCS) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
  }
  __syncthreads();
  if (CG == 2) pair_sync();  // everything the pair sends each other has arrived
  if (warp == 1) {
    tc_fence_after();
    free_tmem<CG>(tmem_base, C::TMEM_COLS);
  }
}

// Adds the partial accumulators of every tile that was cut (at most MAX_PIECES) and applies the epilogue. Item: one
// row and 8 output columns; grid.x: tiles. With many pieces, SPLIT = 4 threads take every fourth, and are added in
// a fixed order (the block's forward, T = 115, H = 2432, F = 12440, 10 tiles in 7 pieces each: 53.2 us by four, 55.6 by
// one; T = 333, H = 2056, F = 5464, 34 tiles in 2: 47.0 by four, 45.1 by one).
constexpr int FIX_THREADS = 256;
constexpr int MAX_PIECES = 16, MANY_PIECES = 6;
template <int OP, int CG, int BN, int SPLIT>
__global__ void __launch_bounds__(FIX_THREADS) fixup_kernel(const __grid_constant__ Params p) {
  constexpr bool GATEUP = is_gateup(OP), QUANT = OP == OP_GATEUP_MX;
  constexpr int NV = GATEUP ? 16 : 8, FIX_ITEMS = FIX_THREADS / SPLIT;
  __shared__ float sums[SPLIT > 1 ? SPLIT - 1 : 1][NV][FIX_ITEMS];
  // the activation to be quantised: rows in groups of FIX_ROWS, four items to a 1x32 block
  constexpr int FIX_ROWS = FIX_ITEMS / 4;
  __shared__ float amax[4][FIX_ROWS];
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x / CG, rank = CG == 2 ? (int)blockIdx.x & 1 : 0;
  const int b0 = (int)((long long)i * p.sk_kb / p.sk_per);
  const int b1 = (int)(((long long)i * p.sk_kb + p.KB - 1) / p.sk_per);
  if (b0 == b1) return;  // one CTA (pair) held the whole tile and finished it
  const Origin o = origin<OP, CG, BN>(p, p.n_full + i, rank);
  if (o.rows <= 0) return;
  const int part = threadIdx.x / FIX_ITEMS, item = threadIdx.x % FIX_ITEMS;
  const int groups = (o.rows + FIX_ROWS - 1) / FIX_ROWS;
  const int total = QUANT ? groups * (o.cols / 32) * FIX_ITEMS : (o.cols + 7) / 8 * o.rows;
  for (int e0 = blockIdx.y * FIX_ITEMS; e0 < total; e0 += gridDim.y * FIX_ITEMS) {  // the same for the whole CTA
    const int e = e0 + item, g = e0 / FIX_ITEMS;
    const int r = QUANT ? g % groups * FIX_ROWS + item % FIX_ROWS : e % o.rows;
    const int c = QUANT ? g / groups * 32 + item / FIX_ROWS * 8 : 8 * (e / o.rows);
    const bool ok = e < total && r < o.rows;
    float v[8], u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = u[j] = 0.f;
    if (ok) {
#pragma unroll 4
      for (int b = b0 + part; b <= b1; b += SPLIT) {
        const int slot = 2 * b + (b * p.sk_per > i * p.sk_kb ? 0 : 1);
        const float* src = p.part + (size_t)(slot * CG + rank) * SLOT_FLOATS + (size_t)c * BM + r;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] += src[j * BM];
          if (GATEUP) u[j] += src[(BN / 2 + j) * BM];
        }
      }
    }
    if constexpr (SPLIT > 1) {
      __syncthreads();  // the last round's sums have been read
      if (part > 0)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          sums[part - 1][j][item] = v[j];
          if (GATEUP) sums[part - 1][(NV - 8) + j][item] = u[j];
        }
      __syncthreads();
      if (part == 0)
#pragma unroll
        for (int s = 0; s < SPLIT - 1; ++s)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            v[j] += sums[s][j][item];
            if (GATEUP) u[j] += sums[s][(NV - 8) + j][item];
          }
    }
    const long long row = o.m0 + r;
    if constexpr (QUANT) {
      float am = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = swiglu::act(v[j], u[j]);
        am = fmaxf(am, fabsf(v[j]));
      }
      __syncthreads();  // the last round's have been read
      if (part == 0) amax[item / FIX_ROWS][item % FIX_ROWS] = am;
      __syncthreads();
      if (part > 0 || !ok) continue;
      const int l = item % FIX_ROWS;
      const uint8_t sb = ggmx::mx_scale_byte(fmaxf(fmaxf(amax[0][l], amax[1][l]), fmaxf(amax[2][l], amax[3][l])));
      const float inv = ggmx::mx_inv_scale(sb);
      uint32_t w[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        w[k] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[4 * k] * inv, v[4 * k + 1] * inv), __NV_SATFINITE,
                                                  __NV_E4M3) |
               (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[4 * k + 2] * inv, v[4 * k + 3] * inv), __NV_SATFINITE,
                                                  __NV_E4M3)
                   << 16;
      const long long at = row * p.ldc + o.n0 + c;
      *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(p.C) + at) = make_uint2(w[0], w[1]);
      if (item / FIX_ROWS == 0) p.C_sf[at >> 5] = sb;
      continue;
    }
    if (part > 0 || !ok) continue;
    const auto pack = [](const float (&t)[8]) {
      return make_uint4(pack_bf16x2(t[0], t[1]), pack_bf16x2(t[2], t[3]), pack_bf16x2(t[4], t[5]),
                        pack_bf16x2(t[6], t[7]));
    };
    if constexpr (OP == OP_GATEUP) {
      if (p.save_hi) {
        const long long at = row * p.ld2 + o.n0 + c;
        const auto keep = [&](long long x, const float (&f)[8]) {
          *reinterpret_cast<uint4*>(p.save_hi + x) = make_uint4(swiglu::hi2(f[0], f[1]), swiglu::hi2(f[2], f[3]),
                                                                swiglu::hi2(f[4], f[5]), swiglu::hi2(f[6], f[7]));
          *reinterpret_cast<uint2*>(p.save_lo + x) =
              make_uint2(swiglu::lo4(f[0], f[1], f[2], f[3]), swiglu::lo4(f[4], f[5], f[6], f[7]));
        };
        keep(at, v);
        keep(at + p.up, u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = swiglu::act(v[j], u[j]);
      *reinterpret_cast<uint4*>(p.C + row * p.ldc + o.n0 + c) = pack(v);
    } else if constexpr (OP == OP_DGRAD_ACT) {
      const long long at = row * p.ld2 + o.n0 + c;
      float zg[8], zu[8];
      const auto get = [&](long long x, float (&f)[8]) {
        const uint4 hi = *reinterpret_cast<const uint4*>(p.save_hi + x);
        const uint2 lo = *reinterpret_cast<const uint2*>(p.save_lo + x);
        swiglu::join4(hi.x, hi.y, lo.x, *reinterpret_cast<float(*)[4]>(&f[0]));
        swiglu::join4(hi.z, hi.w, lo.y, *reinterpret_cast<float(*)[4]>(&f[4]));
      };
      get(at, zg);
      get(at + p.up, zu);
#pragma unroll
      for (int j = 0; j < 8; ++j) swiglu::grad(v[j], zg[j], zu[j], v[j], u[j]);
      *reinterpret_cast<uint4*>(p.C + at) = pack(v);
      *reinterpret_cast<uint4*>(p.C + at + p.up) = pack(u);
    } else {
      *reinterpret_cast<uint4*>((o.second ? p.C2 : p.C) + row * p.ldc + o.n0 + c) = pack(v);
    }
  }
}

// Launch with programmatic dependence on the kernel before it in the stream (every kernel here waits for it).
template <class K>
int launch_dep(K kern, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st, const Params& p, bool dep) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  int n = 0;
  if (dep) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster;
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

// Pairs of CTAs that can be resident at once on the current device.
template <int OP>
int max_pairs() {
  static std::atomic<int> cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    (void)cudaGetLastError();
    return 0;
  }
  if (!cached[dev]) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * (MAX_CTAS / 2));
    cfg.blockDim = dim3(Cfg<OP, 2, 256>::THREADS);
    cfg.dynamicSmemBytes = Cfg<OP, 2, 256>::SMEM_BYTES;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(gemm_kernel<OP, 2, 256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<OP, 2, 256>::SMEM_BYTES) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, gemm_kernel<OP, 2, 256>, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      n = 0;
    }
    cached[dev] = n > 0 ? n : -1;
  }
  return std::max(cached[dev].load(), 0);
}

// Form and work split of a product, chosen before its tensor maps are made (the form sets the boxes of B).
struct Plan {
  int cg, bn;
  int workers;  // CTAs (pairs)
  int b_box;    // rows of a K-major B box
};

// Order of the tiles: the smaller operand stays in L2 while the other streams by; one too large for that goes in groups
// of panels (T = 16384, H = 4096, F = 14336, the block's forward: 5400 us m first, 4900 the smaller first, 4290 in
// groups; MXFP8, H = F = 8192: 3315, 3175, 2865; a training step of T = 4096: 3550, 3310 and, with everything in
// groups, 3380).
constexpr long long L2_KEEP = 48ll << 20;
constexpr int GROUP_ROWS = 2048;

// The form of least estimated time: rounds of tiles times k-blocks times a k-block's time, measured in us (down
// projection, T = H = F = 4096, all in one launch: 97.9 us with one CTA and 256 columns, 109.0 with 128, pairs 82.1 and
// 91.2, MXFP8 57.4, 63.8, 49.8 and 57.9; 24 k-blocks of T = 1001, H = 2048: 14.4, 11.6, 14.4 and 12.3). Cutting the
// tiles of the last round along K saves the idle part of that round and costs partial sums out and in again and one
// more kernel: where every CTA has one piece 4 us for 2 pieces a tile to 8 for 8, and half as much again to twice that
// where its rows are all there (MXFP8 gate/up, H = 7168, F = 2048, 32 tokens, one CTA and 128 columns: 18.5 us whole,
// 16.0 in 2 pieces, 14.4 in 4; 128 tokens: 20.5, 18.5 and 19.1; down, H = 4096, F = 14336, 128 tokens: 55.8, 38.9 and
// 32.6). A rest of more than half a round cannot be cut so; there the line of its k-blocks is cut into equal pieces, of
// which most CTAs have two (13 us). A pair takes 1 us more to set up and to leave.
template <int OP>
Plan plan_for(Params& p, int sms, int pairs) {
  static constexpr float KB_US[2][2][2] = {{{0.22f, 0.355f}, {0.185f, 0.29f}},   // bf16: [pairs][256 columns]
                                           {{0.25f, 0.38f}, {0.22f, 0.335f}}};    // MXFP8
  sms = std::min(sms, MAX_CTAS);
  pairs = std::min(pairs, sms / 2);
  Plan c{};
  float best = 1e30f;
  for (int cg = 1; cg <= 2; ++cg) {
    const int workers = cg == 2 ? pairs : sms;
    if (workers == 0) continue;
    const int per = (p.M + BM * cg - 1) / (BM * cg), tiles_m = p.halves * per;
    for (int bn = 128; bn <= 256; bn *= 2) {
      const int step = is_gateup(OP) ? bn / 2 : bn;
      const int tiles_n = (p.N + step - 1) / step;
      const long long total = (long long)tiles_m * tiles_n, rounds = total / workers;
      const int rest = (int)(total % workers);
      const float kb = KB_US[is_mx(OP)][cg - 1][bn / 256];
      const auto take = [&](float us, int cut, int sk_per, int sk_kb) {
        if (us >= best) return;
        best = us;
        c = {cg, bn, workers, is_gateup(OP) ? bn / 2 : std::min(128, bn / cg)};
        p.tiles_m = tiles_m;
        p.tm_split = per;
        p.tiles_n = tiles_n;
        p.n_full = (int)(total - cut);
        p.sk_tiles = cut;
        p.sk_per = sk_per;
        p.sk_kb = sk_kb;
      };
      const float filled = (float)p.M / (per * BM * cg), fix = cg == 2 ? 1.f : 0.f;
      take((rounds + (rest ? 1 : 0)) * p.KB * kb + fix, 0, 0, p.KB);
      for (int n = 2; rest > 0 && n <= MAX_PIECES && rest * n <= workers && n <= p.KB; ++n) {
        const int len = (p.KB + n - 1) / n, used = (p.KB + len - 1) / len;  // pieces of a tile, none empty
        const float join = 3.f + 0.6f * used + filled * (2.f + 0.8f * used);
        take((rounds * p.KB + len) * kb + fix + join, rest, len, len * used);
      }
      if (2 * rest > workers) {
        const int len = (rest * p.KB + workers - 1) / workers;
        take((rounds * p.KB + len) * kb + fix + 13.f, rest, len, p.KB);
      }
    }
  }
  const long long rows_a = (long long)p.M * p.halves, rows_b = (long long)p.N * (is_gateup(OP) ? 2 : 1);
  p.n_fast = rows_b < rows_a;
  const int fast = p.n_fast ? p.tiles_n : p.tiles_m;
  p.group = std::min(rows_a, rows_b) * p.KB * 128 > L2_KEEP ? std::min(fast, GROUP_ROWS / (BM * c.cg)) : fast;
  return c;
}

template <int OP>
Plan plan(Params& p) {
  return plan_for<OP>(p, moe_host::num_sms(), max_pairs<OP>());
}

template <int OP, int CG, int BN>
int launch_form(const Params& p, int workers, cudaStream_t st, bool dep) {
  using C = Cfg<OP, CG, BN>;
  auto kern = gemm_kernel<OP, CG, BN>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  int n = std::min(p.n_full, workers);
  if (p.sk_tiles) n = std::max(n, (p.sk_tiles * p.sk_kb + p.sk_per - 1) / p.sk_per);
  int rc = launch_dep(kern, dim3(n * CG), C::THREADS, C::SMEM_BYTES, CG, st, p, dep);
  if (rc || !p.sk_tiles) return rc;
  const int per_tile = BM * C::N_STEP / 8 / FIX_THREADS;  // CTAs, one item per thread
  if (p.KB > MANY_PIECES * p.sk_per)
    return launch_dep(fixup_kernel<OP, CG, BN, 4>, dim3(p.sk_tiles * CG, 4 * per_tile), FIX_THREADS, 0, 1, st, p, true);
  return launch_dep(fixup_kernel<OP, CG, BN, 1>, dim3(p.sk_tiles * CG, per_tile), FIX_THREADS, 0, 1, st, p, true);
}

// dep: the kernel before it in the stream is one of the same call's.
template <int OP>
int launch(const Params& p, const Plan& c, cudaStream_t st, bool dep) {
  if (c.cg == 2)
    return c.bn == 256 ? launch_form<OP, 2, 256>(p, c.workers, st, dep) : launch_form<OP, 2, 128>(p, c.workers, st, dep);
  return c.bn == 256 ? launch_form<OP, 1, 256>(p, c.workers, st, dep) : launch_form<OP, 1, 128>(p, c.workers, st, dep);
}

}  // namespace dense
