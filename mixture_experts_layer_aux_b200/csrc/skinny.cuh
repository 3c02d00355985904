// skinny.cuh -- the gated feed-forward block for few tokens (one token of a
// decoding step up to 8 NT), where the time is that of streaming the weights
// once. The weights are the M side of mma.sync (16 rows), the tokens its N side
// (8 per fragment), so nothing is padded to a 128-token tile:
//   gate/up  a CTA owns 8 columns f of F: its 16 weight rows are W_g[f..f+7]
//            and W_u[f..f+7], so gate and up of one element end in the same
//            place and the SwiGLU is applied in the same kernel;
//   down     a CTA owns 16 rows of W_d.
// The W warps of a CTA split K in interleaved runs of 128 elements; their
// partial sums (fp32) are added in warp order through shared memory.
//
// Operands come straight from global memory into the MMA fragments. K may be
// permuted inside a fragment as long as both operands agree: thread t of a
// quad takes 8 consecutive elements of a 32-wide chunk (16 bytes of bf16), and
// the two K16 steps of the chunk are its first and last four. The next run's
// loads are issued before the current run's MMAs.
//
// MXFP8: the codes are widened to f16, exactly; each 1x32 block is one chunk,
// whose fp32 dot product is multiplied by the two blocks' scales.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "gemm_mx.cuh"

namespace skinny {

constexpr int MAX_NT = 4;
constexpr int MAX_T = 8 * MAX_NT;
constexpr int RUN = 128;  // elements of K per warp step

struct Params {
  const uint8_t* W0;     // W_g or W_d, row-major [N, K]
  const uint8_t* W1;     // W_u
  const uint8_t* sf0;    // MXFP8: ue8m0 [N, K/32]
  const uint8_t* sf1;
  const uint8_t* x;      // [T, K]
  const uint8_t* x_sf;   // MXFP8: [T, K/32]
  void* out;             // gate/up: a [T, N] (bf16, or e4m3 codes); down: y [T, N] bf16
  uint8_t* out_sf;       // MXFP8 gate/up: [T, N/32]
  __nv_bfloat16* save;   // bf16 gate/up: gate | up [T, 2N], or NULL
  int T, N, K;
};

MOE_DEV void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
MOE_DEV void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                           uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights are read once: no L1 allocation.
MOE_DEV uint4 ld_w16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
MOE_DEV uint2 ld_w8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// Two e4m3 codes (low half of w) -> f16x2, exact.
MOE_DEV uint32_t e4m3x2_f16(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
// 2^(b - 127); byte 0 is 2^-127 (subnormal), byte 255 is NaN.
MOE_DEV float ue8m0(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
}

// ---------------------------------------------------------------- operand runs

struct Bf16 {
  static constexpr int EB = 2;                                         // bytes per element
  static constexpr int CHUNKS = 4;                                     // 32-wide chunks per run
  template <int NT>
  struct Run {
    uint4 w[CHUNKS][2];
    uint4 x[CHUNKS][NT];
  };
  template <int NT>
  MOE_DEV static void load_w(Run<NT>& r, const uint8_t* p0, const uint8_t* p1, const uint8_t*, const uint8_t*, int k,
                             int K, bool ok0, bool ok1) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int kk = k + 32 * c + 8 * t;  // K % 8 == 0: a thread's eight elements exist or do not
      const bool in = kk < K;
      r.w[c][0] = in && ok0 ? ld_w16(p0 + 2LL * kk) : make_uint4(0, 0, 0, 0);
      r.w[c][1] = in && ok1 ? ld_w16(p1 + 2LL * kk) : make_uint4(0, 0, 0, 0);
    }
  }
  template <int NT>
  MOE_DEV static void load_x(Run<NT>& r, const Params& p, int k) {
    const int t = threadIdx.x & 3, g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int kk = k + 32 * c + 8 * t;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int tok = 8 * n + g;
        r.x[c][n] = kk < p.K && tok < p.T
                        ? *reinterpret_cast<const uint4*>(p.x + 2LL * ((long long)tok * p.K + kk))
                        : make_uint4(0, 0, 0, 0);
      }
    }
  }
  template <int NT>
  MOE_DEV static void mma(const Run<NT>& r, float (&acc)[NT][4]) {
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_bf16_16816(acc[n], r.w[c][0].x, r.w[c][1].x, r.w[c][0].y, r.w[c][1].y, r.x[c][n].x, r.x[c][n].y);
        mma_bf16_16816(acc[n], r.w[c][0].z, r.w[c][1].z, r.w[c][0].w, r.w[c][1].w, r.x[c][n].z, r.x[c][n].w);
      }
  }
};

struct Mx {
  static constexpr int EB = 1;
  static constexpr int CHUNKS = 4;
  template <int NT>
  struct Run {
    uint2 w[CHUNKS][2];
    uint2 x[CHUNKS][NT];
    uint32_t s[2];   // the four blocks' scale bytes of the two weight rows
    uint32_t xs[NT];  // of this thread's token (g) of each fragment
  };
  template <int NT>
  MOE_DEV static void load_w(Run<NT>& r, const uint8_t* p0, const uint8_t* p1, const uint8_t* s0, const uint8_t* s1,
                             int k, int K, bool ok0, bool ok1) {
    const int t = threadIdx.x & 3;
    const bool in = k < K;  // K % 128 == 0: whole runs
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      const int kk = k + 32 * c + 8 * t;
      r.w[c][0] = in && ok0 ? ld_w8(p0 + kk) : make_uint2(0, 0);
      r.w[c][1] = in && ok1 ? ld_w8(p1 + kk) : make_uint2(0, 0);
    }
    r.s[0] = in && ok0 ? __ldg(reinterpret_cast<const uint32_t*>(s0 + k / 32)) : 0u;
    r.s[1] = in && ok1 ? __ldg(reinterpret_cast<const uint32_t*>(s1 + k / 32)) : 0u;
  }
  template <int NT>
  MOE_DEV static void load_x(Run<NT>& r, const Params& p, int k) {
    const int t = threadIdx.x & 3, g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int tok = 8 * n + g;
      const bool in = k < p.K && tok < p.T;
#pragma unroll
      for (int c = 0; c < CHUNKS; ++c)
        r.x[c][n] = in ? *reinterpret_cast<const uint2*>(p.x + (long long)tok * p.K + k + 32 * c + 8 * t)
                       : make_uint2(0, 0);
      r.xs[n] = in ? *reinterpret_cast<const uint32_t*>(p.x_sf + (long long)tok * (p.K / 32) + k / 32) : 0u;
    }
  }
  template <int NT>
  MOE_DEV static void mma(const Run<NT>& r, float (&acc)[NT][4]) {
    const int t = threadIdx.x & 3;
    uint32_t xs0[NT], xs1[NT];  // scale words of tokens 2t and 2t + 1, the columns of this thread's accumulators
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      xs0[n] = __shfl_sync(0xffffffffu, r.xs[n], 8 * t);
      xs1[n] = __shfl_sync(0xffffffffu, r.xs[n], 8 * t + 4);
    }
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      uint32_t a[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i][0] = e4m3x2_f16(r.w[c][i].x);
        a[i][1] = e4m3x2_f16(r.w[c][i].x >> 16);
        a[i][2] = e4m3x2_f16(r.w[c][i].y);
        a[i][3] = e4m3x2_f16(r.w[c][i].y >> 16);
      }
      const float s0 = ue8m0((r.s[0] >> (8 * c)) & 0xffu), s1 = ue8m0((r.s[1] >> (8 * c)) & 0xffu);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        const uint2 x = r.x[c][n];
        mma_f16_16816(d, a[0][0], a[1][0], a[0][1], a[1][1], e4m3x2_f16(x.x), e4m3x2_f16(x.x >> 16));
        mma_f16_16816(d, a[0][2], a[1][2], a[0][3], a[1][3], e4m3x2_f16(x.y), e4m3x2_f16(x.y >> 16));
        const float y0 = ue8m0((xs0[n] >> (8 * c)) & 0xffu), y1 = ue8m0((xs1[n] >> (8 * c)) & 0xffu);
        // the weight's scale first: a block's dot product is at most 32 * 448^2, so neither step overflows
        // unless the block's value itself does
        acc[n][0] += d[0] * s0 * y0;
        acc[n][1] += d[1] * s0 * y1;
        acc[n][2] += d[2] * s1 * y0;
        acc[n][3] += d[3] * s1 * y1;
      }
    }
  }
};

// ---------------------------------------------------------------- kernel

MOE_DEV uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
MOE_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
MOE_DEV void st_cluster(const void* local, uint32_t rank, float v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(local)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// FMT: Bf16 or Mx. GATEUP: rows 0..7 of the tile are W_g[f0..], rows 8..15 W_u[f0..]; else rows n0..n0+15 of W0.
// An MXFP8 gate/up launch runs in clusters of four CTAs, whose 32 columns are one block of the activation's
// quantisation: the CTAs exchange their maxima through distributed shared memory.
template <class FMT, int NT, bool GATEUP, int W>
__global__ void __launch_bounds__(32 * W) gemm_kernel(const Params p) {
  __shared__ float red[W][16][8 * NT + 1];
  __shared__ float cmax[4][8 * NT];
  constexpr bool MXQ = GATEUP && FMT::EB == 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * (GATEUP ? 8 : 16);
  const int r0 = n0 + g, r1 = GATEUP ? n0 + g : n0 + g + 8;
  const bool ok0 = r0 < p.N, ok1 = r1 < p.N;
  const uint8_t* p0 = p.W0 + (long long)r0 * p.K * FMT::EB;
  const uint8_t* p1 = (GATEUP ? p.W1 : p.W0) + (long long)r1 * p.K * FMT::EB;
  const uint8_t* s0 = p.sf0 + (long long)r0 * (p.K / 32);
  const uint8_t* s1 = (GATEUP ? p.sf1 : p.sf0) + (long long)r1 * (p.K / 32);

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  typename FMT::template Run<NT> cur, nxt;
  int k = warp * RUN;
  // the first weights do not depend on the kernel before this one: they are on their way while it ends
  FMT::template load_w<NT>(cur, p0, p1, s0, s1, k, p.K, ok0, ok1);
  griddep_wait();
  griddep_launch_dependents();
  FMT::template load_x<NT>(cur, p, k);
  for (; k < p.K; k += W * RUN) {
    const int kn = k + W * RUN;
    if (kn < p.K) {  // warp-uniform
      FMT::template load_w<NT>(nxt, p0, p1, s0, s1, kn, p.K, ok0, ok1);
      FMT::template load_x<NT>(nxt, p, kn);
    }
    FMT::template mma<NT>(cur, acc);
    cur = nxt;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    red[warp][g][8 * n + 2 * t] = acc[n][0];
    red[warp][g][8 * n + 2 * t + 1] = acc[n][1];
    red[warp][g + 8][8 * n + 2 * t] = acc[n][2];
    red[warp][g + 8][8 * n + 2 * t + 1] = acc[n][3];
  }
  __syncthreads();
  if constexpr (GATEUP) {
    constexpr int ITEMS = 8 * 8 * NT;  // (token, column): column fastest
    constexpr int PER = (ITEMS + 32 * W - 1) / (32 * W);
    float a[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = threadIdx.x + i * 32 * W;
      const int tok = e >> 3, f = e & 7;
      a[i] = 0.f;
      if (e < ITEMS) {
        float gv = 0.f, uv = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          gv += red[w][f][tok];
          uv += red[w][f + 8][tok];
        }
        a[i] = silu_f(gv) * uv;
        if constexpr (!MXQ) {
          if (tok < p.T && n0 + f < p.N) {
            reinterpret_cast<__nv_bfloat16*>(p.out)[(long long)tok * p.N + n0 + f] = __float2bfloat16_rn(a[i]);
            if (p.save) {
              __nv_bfloat16* sv = p.save + (long long)tok * 2 * p.N + n0 + f;
              sv[0] = __float2bfloat16_rn(gv);
              sv[p.N] = __float2bfloat16_rn(uv);
            }
          }
        }
      }
      if constexpr (MXQ) {
        float am = fabsf(a[i]);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        if (e < ITEMS && f < 4) st_cluster(&cmax[cluster_rank()][tok], f, am);
      }
    }
    if constexpr (MXQ) {
      cluster_sync();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = threadIdx.x + i * 32 * W;
        const int tok = e >> 3, f = e & 7;
        if (e < ITEMS && tok < p.T) {
          const float am = fmaxf(fmaxf(cmax[0][tok], cmax[1][tok]), fmaxf(cmax[2][tok], cmax[3][tok]));
          const uint8_t sb = ggmx::mx_scale_byte(am);
          reinterpret_cast<uint8_t*>(p.out)[(long long)tok * p.N + n0 + f] =
              __nv_cvt_float_to_fp8(a[i] * ggmx::mx_inv_scale(sb), __NV_SATFINITE, __NV_E4M3);
          if (f == 0 && cluster_rank() == 0) p.out_sf[(long long)tok * (p.N / 32) + n0 / 32] = sb;
        }
      }
    }
  } else {
    constexpr int ITEMS = 16 * 8 * NT;
    for (int e = threadIdx.x; e < ITEMS; e += 32 * W) {
      const int tok = e >> 4, r = e & 15;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v += red[w][r][tok];
      if (tok < p.T && n0 + r < p.N)
        reinterpret_cast<__nv_bfloat16*>(p.out)[(long long)tok * p.N + n0 + r] = __float2bfloat16_rn(v);
    }
  }
}

template <class FMT, int NT, bool GATEUP, int W>
int launch_nt(const Params& p, cudaStream_t st, bool dep) {
  constexpr bool MXQ = GATEUP && FMT::EB == 1;
  cudaLaunchConfig_t cfg{};
  const int per = GATEUP ? 8 : 16;
  cfg.gridDim = dim3((p.N + per - 1) / per);
  cfg.blockDim = dim3(32 * W);
  cfg.stream = st;
  cudaLaunchAttribute at[2] = {};
  int n = 0;
  if (dep) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (MXQ) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = 4;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  if (cudaLaunchKernelEx(&cfg, gemm_kernel<FMT, NT, GATEUP, W>, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

// dep: the kernel before it in the stream is one of the same call's (the weights are not its results).
template <class FMT, bool GATEUP>
int launch(const Params& p, cudaStream_t st, bool dep) {
  constexpr int W = 8;
  if (p.T <= 8) return launch_nt<FMT, 1, GATEUP, W>(p, st, dep);
  if (p.T <= 16) return launch_nt<FMT, 2, GATEUP, W>(p, st, dep);
  return launch_nt<FMT, 4, GATEUP, W>(p, st, dep);
}

}  // namespace skinny
