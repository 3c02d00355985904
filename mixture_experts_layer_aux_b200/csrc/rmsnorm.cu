// rmsnorm.cu -- root-mean-square norm of the residual stream, forward and
// backward: the norm that makes the layer's x. Forward, per row of H:
//   h = x + residual,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w,
// y in bf16 (the router's and BF16 experts' operand) and/or MXFP8 (the MXFP8
// operands' 1x32 blocks along H, quantised from the fp32 y). Backward, with
// xhat = h rstd and g = w dy:
//   dx = dh + rstd (g - xhat mean(g xhat)),  dweight = sum_t dy xhat.
//
// Both are bound by memory: a row is read once, held in registers (V vectors
// of 8 bf16 per thread), reduced with one block barrier and written once.
// Of the backward this holds up to H = 8192 (8192 rows with dh: H = 4096 49 us,
// 7168 85, 8192 94, 0.83 to 0.88 of the copy's rate). With V = 4 the row, the next
// one and the weight gradient are more than the registers hold: 200 bytes a
// thread, 400 with dh, go through local memory, and one CTA fits an SM
// (H = 12288 301 us, 16384 358, 0.41 and 0.46).
// CTAs are persistent over rows, so the weight stays in registers and the next
// row's loads are in flight while the current row is reduced and written. Rows
// are counted unsigned: T goes up to 2^31 - 1, and a CTA's next row passes it.
#include "common.cuh"
#include "gemm_mx.cuh"
#include "layout.h"

namespace rms {

constexpr int MAX_THREADS = 512;
constexpr int MAX_H = 16384;  // MAX_THREADS x 4 vectors of 8
// CTAs of the backward, each of which leaves one row of partial dweight: two per SM of a B200. A constant, so that
// the workspace does not depend on the device that is current.
constexpr int BWD_CTAS = 2 * 148;

MOE_DEV uint4 ld_stream(const __nv_bfloat16* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }
// bf16 pair -> fp32 is a shift: element 2i in the low half of word i
MOE_DEV float lo(uint32_t w) { return __uint_as_float(w << 16); }
MOE_DEV float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
MOE_DEV float elem(const uint4& u, int i) {
  const uint32_t w = i < 2 ? u.x : i < 4 ? u.y : i < 6 ? u.z : u.w;
  return (i & 1) ? hi(w) : lo(w);
}
MOE_DEV uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// Sum over the block, in a fixed order, one barrier: `buf` alternates between calls, so that a call's writes
// never meet the reads of the call before it.
MOE_DEV float block_sum(float s, float* buf, int nwarp) {
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (nwarp == 1) return s;
  if (lane == 0) buf[warp] = s;
  __syncthreads();
  s = lane < nwarp ? buf[lane] : 0.f;
#pragma unroll
  for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);  // nwarp <= 16
  return __shfl_sync(0xffffffffu, s, 0);
}

struct FwdParams {
  const __nv_bfloat16* x;
  const __nv_bfloat16* res;
  const __nv_bfloat16* w;
  __nv_bfloat16* h;
  __nv_bfloat16* y;
  uint8_t* q;
  uint8_t* sf;
  float* rstd;
  int T, H;
  float eps;
};

template <int V, bool RES>
__global__ void __launch_bounds__(MAX_THREADS) fwd_kernel(const FwdParams p) {
  __shared__ float red[2][16];
  const int nvec = p.H >> 3;
  const int nwarp = blockDim.x >> 5;
  uint4 w[V], cx[V], cr[V];
  bool ok[V];
  auto load = [&](uint32_t row, uint4 (&a)[V], uint4 (&b)[V]) {
    const long long base = (long long)row * p.H;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      a[i] = ok[i] ? ld_stream(p.x + base + 8LL * c) : make_uint4(0, 0, 0, 0);
      if (RES) b[i] = ok[i] ? ld_stream(p.res + base + 8LL * c) : make_uint4(0, 0, 0, 0);
    }
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    ok[i] = c < nvec;
    w[i] = ok[i] ? *reinterpret_cast<const uint4*>(p.w + 8LL * c) : make_uint4(0, 0, 0, 0);
  }
  load(blockIdx.x, cx, cr);
  int flip = 0;
  for (uint32_t row = blockIdx.x; row < (uint32_t)p.T; row += gridDim.x) {
    float v[V][8];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = elem(cx[i], j);
        if (RES) v[i][j] += elem(cr[i], j);
        ss += v[i][j] * v[i][j];
      }
    // the next row's loads go out before this row's reduction
    if (row + gridDim.x < (uint32_t)p.T) load(row + gridDim.x, cx, cr);
    const float sum = block_sum(ss, red[flip], nwarp);
    flip ^= 1;
    const float rstd = __frsqrt_rn(sum / (float)p.H + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
    const long long base = (long long)row * p.H;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (p.h && ok[i]) *reinterpret_cast<uint4*>(p.h + base + 8LL * c) = pack8(v[i]);
      float am = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = v[i][j] * rstd * elem(w[i], j);
        am = fmaxf(am, fabsf(v[i][j]));
      }
      if (p.y && ok[i]) *reinterpret_cast<uint4*>(p.y + base + 8LL * c) = pack8(v[i]);
      if (p.q) {
        // a 1x32 block is the 8 elements of four consecutive lanes (H % 32 == 0: all four in the row, or none)
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
        am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
        const uint8_t sb = ggmx::mx_scale_byte(am);
        const float inv = ggmx::mx_inv_scale(sb);
        uint32_t code[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const __nv_fp8x2_storage_t a = __nv_cvt_float2_to_fp8x2(
              make_float2(v[i][4 * k] * inv, v[i][4 * k + 1] * inv), __NV_SATFINITE, __NV_E4M3);
          const __nv_fp8x2_storage_t b = __nv_cvt_float2_to_fp8x2(
              make_float2(v[i][4 * k + 2] * inv, v[i][4 * k + 3] * inv), __NV_SATFINITE, __NV_E4M3);
          code[k] = (uint32_t)a | ((uint32_t)b << 16);
        }
        if (ok[i]) {
          *reinterpret_cast<uint2*>(p.q + base + 8LL * c) = make_uint2(code[0], code[1]);
          if ((threadIdx.x & 3) == 0) p.sf[(base >> 5) + (c >> 2)] = sb;
        }
      }
    }
  }
}

struct BwdParams {
  const __nv_bfloat16* dy;
  const __nv_bfloat16* h;
  const __nv_bfloat16* w;
  const float* rstd;
  const __nv_bfloat16* dh;
  __nv_bfloat16* dx;
  float* part;  // [gridDim.x, H] partial dweight, or NULL
  int T, H;
};

template <int V, bool DH>
__global__ void __launch_bounds__(MAX_THREADS) bwd_kernel(const BwdParams p) {
  __shared__ float red[2][16];
  const int nvec = p.H >> 3;
  const int nwarp = blockDim.x >> 5;
  griddep_launch_dependents();
  uint4 w[V], ny[V], nh[V], nd[V];
  float nr;
  bool ok[V];
  float dw[V][8];
  auto load = [&](uint32_t row) {
    const long long base = (long long)row * p.H;
    nr = p.rstd[row];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const long long c = base + 8LL * (threadIdx.x + i * blockDim.x);
      ny[i] = ok[i] ? ld_stream(p.dy + c) : make_uint4(0, 0, 0, 0);
      nh[i] = ok[i] ? ld_stream(p.h + c) : make_uint4(0, 0, 0, 0);
      if (DH) nd[i] = ok[i] ? ld_stream(p.dh + c) : make_uint4(0, 0, 0, 0);
    }
  };
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    ok[i] = c < nvec;
    w[i] = ok[i] ? *reinterpret_cast<const uint4*>(p.w + 8LL * c) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  }
  load(blockIdx.x);
  int flip = 0;
  for (uint32_t row = blockIdx.x; row < (uint32_t)p.T; row += gridDim.x) {
    uint4 cy[V], ch[V], cd[V];
    const float r = nr;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      cy[i] = ny[i];
      ch[i] = nh[i];
      if (DH) cd[i] = nd[i];
    }
    if (row + gridDim.x < (uint32_t)p.T) load(row + gridDim.x);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = elem(cy[i], j), xh = elem(ch[i], j) * r;
        dot += d * elem(w[i], j) * xh;
        dw[i][j] += d * xh;
      }
    const float c1 = block_sum(dot, red[flip], nwarp) / (float)p.H;
    flip ^= 1;
    if (p.dx) {
      const long long base = (long long)row * p.H;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!ok[i]) continue;
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j] = r * (elem(cy[i], j) * elem(w[i], j) - elem(ch[i], j) * r * c1);
          if (DH) o[j] += elem(cd[i], j);
        }
        *reinterpret_cast<uint4*>(p.dx + base + 8LL * (threadIdx.x + i * blockDim.x)) = pack8(o);
      }
    }
  }
  if (p.part) {
    float* part = p.part + (long long)blockIdx.x * p.H;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!ok[i]) continue;
      float4* d = reinterpret_cast<float4*>(part + 8LL * (threadIdx.x + i * blockDim.x));
      d[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      d[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
  }
}

// dweight[c] = sum over the CTAs' partials, in a fixed order: 32 columns per CTA, whose 32 warps take every 32nd
// partial each (at most ten, all loaded at once) before the warps' sums are added.
constexpr int DW_WARPS = 32;
__global__ void __launch_bounds__(32 * DW_WARPS) dweight_kernel(const float* __restrict__ part, int n, int H,
                                                                float* __restrict__ dw) {
  __shared__ float s[DW_WARPS][33];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  constexpr int PER = (BWD_CTAS + DW_WARPS - 1) / DW_WARPS;
  float v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int r = warp + i * DW_WARPS;
    v[i] = c < H && r < n ? part[(long long)r * H + c] : 0.f;
  }
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) a += v[i];
  s[warp][lane] = a;
  __syncthreads();
  // warp w adds column w of the tile
  a = s[lane][warp];
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  if (lane == 0 && blockIdx.x * 32 + warp < H) dw[blockIdx.x * 32 + warp] = a;
}

// Vectors per thread and threads per row.
struct Shape {
  int v, threads;
};
static Shape shape_of(int T, int H, bool bwd) {
  const int nvec = H / 8;
  int v = bwd ? 2 : 4;
  if (T < 148 || nvec < 128) v = 1;  // few rows: spread the row over more threads
  while (nvec > v * MAX_THREADS) v *= 2;
  return {v, ((nvec + v - 1) / v + 31) / 32 * 32};
}

static int bwd_ctas(int T) { return T < BWD_CTAS ? T : BWD_CTAS; }

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static int check(int T, int H) {
  if (T < 1 || H < 1) return MOE_ERR_INVALID_ARG;
  if (H % 8 != 0 || H > MAX_H) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace rms

extern "C" int moe_rmsnorm_fwd(int32_t T, int32_t H, const void* x, const void* residual, const void* weight,
                               float eps, void* h, void* y, uint8_t* y_q, uint8_t* y_sf, float* rstd, void* stream) {
  using namespace rms;
  int rc = check(T, H);
  if (rc) return rc;
  if (!x || !weight || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if ((y_q == nullptr) != (y_sf == nullptr) || (!y && !y_q && !h)) return MOE_ERR_INVALID_ARG;
  if (y_q && H % 32 != 0) return MOE_ERR_UNSUPPORTED;
  if (!al16(x) || !al16(residual) || !al16(weight) || !al16(h) || !al16(y) || !al16(y_q) ||
      (reinterpret_cast<uintptr_t>(rstd) & 3u))
    return MOE_ERR_ALIGNMENT;
  FwdParams p{static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(residual),
              static_cast<const __nv_bfloat16*>(weight), static_cast<__nv_bfloat16*>(h),
              static_cast<__nv_bfloat16*>(y), y_q, y_sf, rstd, T, H, eps};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Shape s = shape_of(T, H, false);
  const int per_sm = s.threads <= 256 ? 512 / s.threads : 1;
  const long long cap = (long long)moe_host::num_sms() * per_sm;
  const int grid = (int)(T < cap ? T : cap);
  auto go = [&](auto kern) { kern<<<grid, s.threads, 0, st>>>(p); };
  if (residual) {
    if (s.v == 1) go(fwd_kernel<1, true>);
    else if (s.v == 2) go(fwd_kernel<2, true>);
    else go(fwd_kernel<4, true>);
  } else {
    if (s.v == 1) go(fwd_kernel<1, false>);
    else if (s.v == 2) go(fwd_kernel<2, false>);
    else go(fwd_kernel<4, false>);
  }
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" size_t moe_rmsnorm_bwd_workspace_size(int32_t T, int32_t H) {
  if (rms::check(T, H)) return 0;
  return ws_round((size_t)rms::bwd_ctas(T) * H * sizeof(float));
}

extern "C" int moe_rmsnorm_bwd(int32_t T, int32_t H, const void* dY, const void* h, const void* weight,
                               const float* rstd, const void* dh, void* dX, float* dweight, void* ws,
                               size_t ws_bytes, void* stream) {
  using namespace rms;
  int rc = check(T, H);
  if (rc) return rc;
  if (!dY || !h || !weight || !rstd || (!dX && !dweight)) return MOE_ERR_INVALID_ARG;
  if (!al16(dY) || !al16(h) || !al16(weight) || !al16(dh) || !al16(dX) || !al16(ws) ||
      ((reinterpret_cast<uintptr_t>(rstd) | reinterpret_cast<uintptr_t>(dweight)) & 3u))
    return MOE_ERR_ALIGNMENT;
  if (dweight && (!ws || ws_bytes < moe_rmsnorm_bwd_workspace_size(T, H))) return MOE_ERR_WORKSPACE;
  BwdParams p{static_cast<const __nv_bfloat16*>(dY), static_cast<const __nv_bfloat16*>(h),
              static_cast<const __nv_bfloat16*>(weight), rstd, static_cast<const __nv_bfloat16*>(dh),
              static_cast<__nv_bfloat16*>(dX), dweight ? static_cast<float*>(ws) : nullptr, T, H};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Shape s = shape_of(T, H, true);
  const int grid = bwd_ctas(T);
  auto go = [&](auto kern) { kern<<<grid, s.threads, 0, st>>>(p); };
  if (dh) {
    if (s.v == 1) go(bwd_kernel<1, true>);
    else if (s.v == 2) go(bwd_kernel<2, true>);
    else go(bwd_kernel<4, true>);
  } else {
    if (s.v == 1) go(bwd_kernel<1, false>);
    else if (s.v == 2) go(bwd_kernel<2, false>);
    else go(bwd_kernel<4, false>);
  }
  MOE_CHECK_LAUNCH();
  if (dweight) {
    // launched while the backward kernel runs; it waits for it
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((H + 31) / 32);
    cfg.blockDim = dim3(32 * DW_WARPS);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, dweight_kernel, (const float*)p.part, grid, (int)H, dweight) != cudaSuccess) {
      (void)cudaGetLastError();
      return MOE_ERR_CUDA;
    }
  }
  return MOE_OK;
}
