// dense.cuh -- dense bf16 GEMM of the gated feed-forward block on the sm_100a
// tensor cores (tcgen05 + TMEM + TMA), any M, and N, K multiples of 8:
//   gate/up   a   = silu(x W_g^T) * (x W_u^T)     (both projections in one tile: [gate | up] columns)
//   down      y   = a W_d^T
//   dgrad     dgu = SwiGLU backward of (dY W_d),  dX = dgate W_g + dup W_u
//   wgrad     dW  = dO^T act
// Everything past an edge of M, N or K is zero-filled by TMA on the way in and
// predicated on the way out, so no operand is padded.
//
// Roles (320 threads, one CTA per SM, persistent), as in the grouped GEMM of
// gemm.cuh: warp 0 TMA producer (four stages of A 128 x 64 and B 256 x 64,
// 128-byte swizzle), warp 1 MMA issuer (M128 N256 K16) and TMEM owner (two
// 256-column accumulators), warps 2..9 epilogue (lane quadrant w % 4, column
// half). Every wait is bounded (MOE_WAIT_NS).
//
// Work split. Whole tiles go round robin over the CTAs while they fill every
// SM; the rest (all tiles, when there are fewer than SMs) is one line of
// k-blocks that is cut into equal pieces, one per CTA. A piece that holds a
// whole tile is finished in place; the others leave fp32 partial accumulators
// in the workspace (at most two per CTA), and fixup_kernel adds them in the
// order of K and applies the epilogue, so results do not depend on timing.
#pragma once

#include "common.cuh"
#include "swiglu.cuh"

namespace dense {

constexpr int BM = 128, BN = 256, BK = 64;
constexpr int kStages = 4;
constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2, STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int NUM_THREADS = 64 + 32 * EPI_WARPS;
constexpr int TMEM_COLS = 2 * BN;
constexpr int STG_ROW = 80;  // staging: 32 rows x (64 + 16) bytes per epilogue warp
constexpr int STG_BYTES = EPI_WARPS * 32 * STG_ROW;
constexpr int BAR_BYTES = 256;
constexpr int SMEM_BYTES = 1024 + kStages * STAGE_BYTES + BAR_BYTES + STG_BYTES;
static_assert(SMEM_BYTES <= 232448, "shared memory");
constexpr int MAX_CTAS = 160;                            // CTAs of one launch (one per SM)
constexpr size_t SLOT_FLOATS = (size_t)BM * BN;          // one partial accumulator
constexpr size_t PART_BYTES = 2ull * MAX_CTAS * SLOT_FLOATS * sizeof(float);

enum Op : int {
  OP_GATEUP = 0,     // A = x, B = W_g | W_u rows (K-major): a, optionally gate/up
  OP_DOWN = 1,       // A, B K-major: bf16
  OP_DGRAD_ACT = 2,  // A = dY K-major, B = W_d MN-major: dgate | dup from the saved gate/up
  OP_DGRAD_X = 3,    // A = dgate then dup (K-major), B = W_g then W_u (MN-major): bf16
  OP_WGRAD = 4,      // A = dO^T, B = act^T (both MN-major): bf16; rows past m_split from A2 into C2
};

struct __align__(64) Params {
  CUtensorMap tmA, tmA2, tmB0, tmB1;
  int M, N;            // output rows and columns (per half when m_split)
  int KB;              // k-blocks of 64
  int kb_split;        // OP_DGRAD_X: k-blocks of the first half
  int tiles_m, tiles_n;
  int tm_split;        // OP_WGRAD: m-tiles of the first half (tiles_m when there is one)
  int n_full;          // tiles done whole, round robin
  int sk_tiles;        // tiles n_full .. n_full + sk_tiles - 1, cut along K
  int sk_per;          // k-blocks per CTA of those
  float* part;
  __nv_bfloat16* C;
  __nv_bfloat16* C2;
  long long ldc;
  __nv_bfloat16* save;            // OP_GATEUP: [M, 2N] gate | up, or NULL
  const __nv_bfloat16* gateup;    // OP_DGRAD_ACT: the same, as saved
  int* status;
};

struct Seg {
  int tile;  // -1: no more
  int kb0, nkb;
  int slot;  // >= 0: partial accumulator to leave there
};

// The it-th piece of work of CTA b: first its cut of the k-block line, then whole tiles.
struct Walk {
  int u, end, t, step;
  MOE_DEV Walk(const Params& p) {
    const int units = p.sk_tiles * p.KB;
    u = min((int)blockIdx.x * p.sk_per, units);
    end = min(u + p.sk_per, units);
    t = blockIdx.x;
    step = gridDim.x;
  }
  MOE_DEV Seg next(const Params& p) {
    Seg s;
    if (u < end) {
      const int i = u / p.KB;
      s.kb0 = u - i * p.KB;
      s.nkb = min(p.KB - s.kb0, end - u);
      s.tile = p.n_full + i;
      s.slot = s.nkb == p.KB ? -1 : 2 * (int)blockIdx.x + (s.kb0 > 0 ? 0 : 1);
      u += s.nkb;
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

template <int OP>
struct Cfg {
  static constexpr bool A_MN = OP == OP_WGRAD;
  static constexpr bool B_MN = OP >= OP_DGRAD_ACT;
  static constexpr int N_STEP = OP == OP_GATEUP ? BN / 2 : BN;  // output columns per tile
};

struct Origin {
  int mt, m0, n0, rows, cols;  // m0, n0 within the (half) output; rows, cols: valid extent
  bool second;                 // OP_WGRAD: the second half
};
template <int OP>
MOE_DEV Origin origin(const Params& p, int tile) {
  Origin o;
  o.mt = tile % p.tiles_m;  // m fastest: the CTAs of a wave share a few column panels of B
  const int nt = tile / p.tiles_m;
  o.second = OP == OP_WGRAD && o.mt >= p.tm_split;
  o.m0 = (o.mt - (o.second ? p.tm_split : 0)) * BM;
  o.n0 = nt * Cfg<OP>::N_STEP;
  o.rows = min(BM, p.M - o.m0);
  o.cols = min(Cfg<OP>::N_STEP, p.N - o.n0);
  return o;
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

MOE_DEV void pack32(const float (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
}
MOE_DEV float word_lo(uint32_t w) { return __uint_as_float(w << 16); }
MOE_DEV float word_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

template <int OP>
__global__ void __launch_bounds__(NUM_THREADS, 1) gemm_kernel(const __grid_constant__ Params p) {
  using C = Cfg<OP>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* stg_area = smem + kStages * STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg_area + STG_BYTES);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // launched over the tail of the kernel before it: its results are visible from here on
  griddep_wait();
  griddep_launch_dependents();

  bool aborted = false;
  Walk walk(p);
  if (warp == 0) {
    // ======================= TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_par = 0;
      for (Seg s = walk.next(p); s.tile >= 0 && !aborted; s = walk.next(p)) {
        const Origin o = origin<OP>(p, s.tile);
        for (int kb = s.kb0; kb < s.kb0 + s.nkb; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status, DEV_WAIT_TIMEOUT_PRODUCER)) {
            aborted = true;
            break;
          }
          mbar_arrive_expect_tx(&full[stage], STAGE_BYTES);
          issued_mask |= 1u << stage;
          issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
          uint8_t* sA = smem + stage * STAGE_BYTES;
          uint8_t* sB = sA + A_BYTES;
          const bool hi = OP == OP_DGRAD_X && kb >= p.kb_split;  // the up half of K
          const int kc = (kb - (hi ? p.kb_split : 0)) * BK;
          const CUtensorMap* mA = (hi || o.second) ? &p.tmA2 : &p.tmA;
          if constexpr (!C::A_MN) {
            tma_load_2d(sA, mA, kc, o.m0, &full[stage]);
          } else {
            tma_load_2d(sA, mA, o.m0, kc, &full[stage]);
            tma_load_2d(sA + 64 * BK * 2, mA, o.m0 + 64, kc, &full[stage]);
          }
          if constexpr (!C::B_MN) {
            tma_load_2d(sB, &p.tmB0, kc, o.n0, &full[stage]);
            if (OP == OP_GATEUP) tma_load_2d(sB + 128 * BK * 2, &p.tmB1, kc, o.n0, &full[stage]);
            else tma_load_2d(sB + 128 * BK * 2, &p.tmB0, kc, o.n0 + 128, &full[stage]);
          } else {
            const CUtensorMap* mB = hi ? &p.tmB1 : &p.tmB0;
#pragma unroll
            for (int j = 0; j < BN / 64; ++j)
              tma_load_2d(sB + j * 64 * BK * 2, mB, o.n0 + 64 * j, kc, &full[stage]);
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (*abort_flag) {
        // every TMA this thread issued must land before the CTA exits
        for (int i = 0; i < kStages; ++i)
          if (issued_mask & (1u << i)) {
            const uint32_t par = (issued_par >> i) & 1u;
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&full[i], par) && globaltimer_ns() - t0 < MOE_WAIT_NS) {
            }
          }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ======================= MMA issuer
    if (lane == 0) {
      constexpr uint32_t IDESC = idesc_bf16(BM, BN, C::A_MN ? 1 : 0, C::B_MN ? 1 : 0);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      for (Seg s = walk.next(p); s.tile >= 0 && !aborted; s = walk.next(p)) {
        if (!mbar_wait(&tempty[acc], acc_phase ^ 1, abort_flag, p.status, DEV_WAIT_TIMEOUT_MMA)) {
          aborted = true;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = 0; kb < s.nkb; ++kb) {
          if (!mbar_wait(&full[stage], phase, abort_flag, p.status, DEV_WAIT_TIMEOUT_MMA)) {
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem + stage * STAGE_BYTES), b0 = a0 + A_BYTES;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ad = C::A_MN ? smem_desc_sw128(a0 + kk * 2048, 64 * BK * 2, 1024)
                                        : smem_desc_sw128(a0 + kk * 32, 16, 1024);
            const uint64_t bd = C::B_MN ? smem_desc_sw128(b0 + kk * 2048, 64 * BK * 2, 1024)
                                        : smem_desc_sw128(b0 + kk * 32, 16, 1024);
            mma_bf16(d_tmem, ad, bd, IDESC, (kb | kk) != 0 ? 1u : 0u);
          }
          mma_commit(&empty[stage]);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (aborted) break;
        mma_commit(&tfull[acc]);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      if (*abort_flag) {
        // wait for every MMA already issued before TMEM is released
        mma_commit(drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < MOE_WAIT_NS) {
        }
      }
    }
    __syncwarp();
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
      const Origin o = origin<OP>(p, s.tile);
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + acc * BN;
      const int rows = o.rows - 32 * q;  // of this warp's 32 (may be <= 0)
      const long long row0 = (long long)o.m0 + 32 * q;
      if (s.slot >= 0) {
        // fp32 partial, column-major: a warp store writes one column's 32 rows
        float* dst = p.part + (size_t)s.slot * SLOT_FLOATS + 32 * q + lane;
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
        const long long ld2 = 2LL * p.N;
#pragma unroll 1
        for (int c = h * 64; c < (h + 1) * 64; c += 32) {
          const int cols = o.cols - c;
          if (cols <= 0) break;  // warp-uniform
          float g[32], u[32];
          uint32_t w[16];
          tmem_ld32(tb + c, g);
          tmem_ld32(tb + BN / 2 + c, u);
          tmem_ld_wait();
          if (p.save) {
            __nv_bfloat16* sv = p.save + row0 * ld2 + o.n0 + c;
            pack32(g, w);
            store_rows(stg, w, sv, ld2, rows, cols);
            pack32(u, w);
            store_rows(stg, w, sv + p.N, ld2, rows, cols);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) g[i] = swiglu::act(g[i], u[i]);
          pack32(g, w);
          store_rows(stg, w, p.C + row0 * p.ldc + o.n0 + c, p.ldc, rows, cols);
        }
      } else if constexpr (OP == OP_DGRAD_ACT) {
        const long long ld2 = 2LL * p.N;
#pragma unroll 1
        for (int c = h * (BN / 2); c < (h + 1) * (BN / 2); c += 32) {
          const int cols = o.cols - c;
          if (cols <= 0) break;
          float v[32];
          uint32_t zg[16], zu[16];
          const __nv_bfloat16* src = p.gateup + row0 * ld2 + o.n0 + c;
          load_rows(stg, zg, src, ld2, rows, cols);
          load_rows(stg, zu, src + p.N, ld2, rows, cols);
          tmem_ld32(tb + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float g0, u0, g1, u1;
            swiglu::grad(v[2 * i], word_lo(zg[i]), word_lo(zu[i]), g0, u0);
            swiglu::grad(v[2 * i + 1], word_hi(zg[i]), word_hi(zu[i]), g1, u1);
            zg[i] = pack_bf16x2(g0, g1);
            zu[i] = pack_bf16x2(u0, u1);
          }
          __nv_bfloat16* dst = p.C + row0 * ld2 + o.n0 + c;
          store_rows(stg, zg, dst, ld2, rows, cols);
          store_rows(stg, zu, dst + p.N, ld2, rows, cols);
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
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1;
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// Adds the partial accumulators of every tile that was cut (in the order of K) and applies the epilogue.
// Thread: one row and 8 output columns; grid.x: tiles, grid.y: column groups of CTA_COLS.
constexpr int FIX_THREADS = 256;
template <int OP>
__global__ void __launch_bounds__(FIX_THREADS) fixup_kernel(const __grid_constant__ Params p) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.x;
  const int b0 = (int)((long long)i * p.KB / p.sk_per), b1 = (int)(((long long)(i + 1) * p.KB - 1) / p.sk_per);
  if (b0 == b1) return;  // one CTA held the whole tile and finished it
  const Origin o = origin<OP>(p, p.n_full + i);
  const int groups = (o.cols + 7) / 8;
  for (int e = blockIdx.y * FIX_THREADS + threadIdx.x; e < groups * o.rows; e += gridDim.y * FIX_THREADS) {
    const int r = e % o.rows, c = 8 * (e / o.rows);
    float v[8], u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = u[j] = 0.f;
    for (int b = b0; b <= b1; ++b) {
      const int slot = 2 * b + (b * p.sk_per > i * p.KB ? 0 : 1);
      const float* src = p.part + (size_t)slot * SLOT_FLOATS + (size_t)c * BM + r;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] += src[j * BM];
        if (OP == OP_GATEUP) u[j] += src[(BN / 2 + j) * BM];
      }
    }
    const long long row = o.m0 + r;
    const auto pack = [](const float (&t)[8]) {
      return make_uint4(pack_bf16x2(t[0], t[1]), pack_bf16x2(t[2], t[3]), pack_bf16x2(t[4], t[5]),
                        pack_bf16x2(t[6], t[7]));
    };
    if constexpr (OP == OP_GATEUP) {
      if (p.save) {
        __nv_bfloat16* sv = p.save + row * 2LL * p.N + o.n0 + c;
        *reinterpret_cast<uint4*>(sv) = pack(v);
        *reinterpret_cast<uint4*>(sv + p.N) = pack(u);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = swiglu::act(v[j], u[j]);
      *reinterpret_cast<uint4*>(p.C + row * p.ldc + o.n0 + c) = pack(v);
    } else if constexpr (OP == OP_DGRAD_ACT) {
      const __nv_bfloat16* src = p.gateup + row * 2LL * p.N + o.n0 + c;
      float zg[8], zu[8];
      unpack_bf16x8(*reinterpret_cast<const uint4*>(src), zg);
      unpack_bf16x8(*reinterpret_cast<const uint4*>(src + p.N), zu);
#pragma unroll
      for (int j = 0; j < 8; ++j) swiglu::grad(v[j], zg[j], zu[j], v[j], u[j]);
      __nv_bfloat16* dst = p.C + row * 2LL * p.N + o.n0 + c;
      *reinterpret_cast<uint4*>(dst) = pack(v);
      *reinterpret_cast<uint4*>(dst + p.N) = pack(u);
    } else {
      *reinterpret_cast<uint4*>((o.second ? p.C2 : p.C) + row * p.ldc + o.n0 + c) = pack(v);
    }
  }
}

// Launch with programmatic dependence on the kernel before it in the stream (every kernel here waits for it).
template <class K>
int launch_dep(K kern, dim3 grid, int threads, size_t smem, cudaStream_t st, const Params& p, bool dep) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = dep ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

// dep: the kernel before it in the stream is one of the same call's.
template <int OP>
int launch(Params& p, cudaStream_t st, bool dep) {
  p.tiles_n = (p.N + Cfg<OP>::N_STEP - 1) / Cfg<OP>::N_STEP;
  const long long total = (long long)p.tiles_m * p.tiles_n;
  int sms = moe_host::num_sms();
  if (sms > MAX_CTAS) sms = MAX_CTAS;
  const int rest = (int)(total % sms);
  p.n_full = (int)(total - rest);
  p.sk_tiles = rest;
  p.sk_per = rest ? (rest * p.KB + sms - 1) / sms : 0;
  auto kern = gemm_kernel<OP>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  int rc = launch_dep(kern, dim3(sms), NUM_THREADS, SMEM_BYTES, st, p, dep);
  if (rc || !rest) return rc;
  return launch_dep(fixup_kernel<OP>, dim3(rest, OP == OP_GATEUP ? 8 : 16), FIX_THREADS, 0, st, p, true);
}

}  // namespace dense
