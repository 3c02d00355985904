// ffn.cu -- the gated feed-forward block y = W_d (silu(W_g x) * (W_u x)) on its
// own (a dense layer of the stack, or a shared expert), forward in bf16 and
// MXFP8 and backward in bf16.
//   few tokens    the streaming kernels of stream.cuh (two launches; MXFP8 from
//                 a bf16 x: three);
//   more          the dense tensor-core kernel of dense.cuh.
// Backward: dgrad of the down projection with the SwiGLU backward in its
// epilogue, the weight gradients, and dX = dgate W_g + dup W_u as one product
// over [dgate | dup].
#include "common.cuh"
#include "dense.cuh"
#include "layout.h"
#include "stream.cuh"

namespace ffn {

using dense::Params;

// Tokens up to which the streaming kernels are taken, whatever the widths: 56 in bf16, 16 in MXFP8. Streaming / dense,
// us:
//   bf16, H x F      48 tokens      56             64
//   8192 x 28672     243  / 264     244  / 258     250  / 251
//   4096 x 14336     75.4 / 75.5    74.6 / 76.3    78.4 / 77.2
//   4096 x 11008     61.9 / 64.7    62.7 / 63.1    64.0 / 65.1
//   2048 x 5504      28.6 / 30.7    30.8 / 30.8    32.6 / 30.6
//   2056 x 5464      32.8 / 31.0    35.6 / 31.9    36.9 / 31.0
//   1024 x 4096      22.5 / 22.5    24.1 / 22.5    24.6 / 20.8
//   MXFP8            16             24             32
//   7168 x 18432     90.7 / 95.3    92.1 / 92.3    92.0 / 88.4
//   4096 x 14336     45.5 / 51.9    49.0 / 52.4    49.2 / 49.2
//   7168 x 2048      22.8 / 30.7    25.9 / 28.2    28.5 / 26.7
//   4096 x 4096      22.5 / 30.4    24.6 / 30.6    27.0 / 28.4
//   1024 x 4096      17.7 / 20.5    20.4 / 20.5    22.3 / 20.6
// So ragged and small widths lose up to 4 us below 57 tokens. In MXFP8, room for 32 tokens in the loader of scales
// (which the figures from 24 on have) costs the calls of fewer 0 to 2 us each: 16 tokens 7168 x 2048 24.5, 8 tokens
// 4096 x 4096 22.4 in place of 20.6.
static bool streams(const moe_ffn_config* c) {
  return c->T <= (c->dtype == MOE_DT_MXFP8 ? stream::MAX_T_MX : stream::MAX_T);
}

#define FFN_RC(x)         \
  do {                    \
    int _rc = (x);        \
    if (_rc) return _rc;  \
  } while (0)

static bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool a4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

static int check_cfg(const moe_ffn_config* c) {
  if (!c) return MOE_ERR_INVALID_ARG;
  if (c->T < 1 || c->H < 1 || c->F < 1) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_DT_BF16 && c->dtype != MOE_DT_MXFP8 && c->dtype != MOE_DT_NVFP4) return MOE_ERR_INVALID_ARG;
  if (c->dtype == MOE_DT_NVFP4) return MOE_ERR_UNSUPPORTED;
  if (c->T > (1 << 24) || c->H > (1 << 20) || c->F > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (c->dtype == MOE_DT_MXFP8) {
    if (c->H % 256 != 0 || c->F % 128 != 0 || c->save_for_bwd) return MOE_ERR_UNSUPPORTED;
  } else if (c->H % 8 != 0 || c->F % 8 != 0) {
    return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

static int cdiv(int a, int b) { return (a + b - 1) / b; }
static int pad64(int n) { return (n + 63) / 64 * 64; }

// A row-major bf16 operand: rows of ld elements.
struct Mat {
  const void* p;
  long long ld;
};

// Rows that do not start on 128 bytes cost more to load (every 128-byte row of a TMA box is on two lines), so the
// buffers of this file are padded to 64 elements. The caller's ragged operands are read as they are: copies with padded
// rows, made once per call, made a training step of T = 4001, H = 4104, F = 8200 2 % faster, but one of T = 2200,
// H = 2056, F = 5464 7 % slower and one of T = 600, H = 4104, F = 8200 17 %.

struct FwdWs {
  __nv_bfloat16* a;  // [T, Fp]
  float* part;
  uint8_t *xq, *xq_sf, *aq, *aq_sf;
};
static size_t carve_fwd(void* ws, const moe_ffn_config* c, FwdWs* w) {
  Carve cv(ws);
  const size_t T = c->T, H = c->H, F = c->F;
  *w = FwdWs{};
  if (c->dtype == MOE_DT_MXFP8) {
    w->xq = cv.take<uint8_t>(T * H);
    w->xq_sf = cv.take<uint8_t>(T * H / 32);
    w->aq = cv.take<uint8_t>(T * F);
    w->aq_sf = cv.take<uint8_t>(T * F / 32);
    if (!streams(c)) w->part = cv.take<float>(dense::PART_BYTES / sizeof(float));
  } else {
    if (!c->save_for_bwd) w->a = cv.take<__nv_bfloat16>(T * pad64(c->F));
    if (!streams(c)) w->part = cv.take<float>(dense::PART_BYTES / sizeof(float));
  }
  return cv.used;
}

// What the backward reads: the pre-activations (24 bits, swiglu.cuh; gate in columns [0, F), up in [Fp, Fp + F) of
// rows of 2 Fp) and the activation.
struct Saved {
  __nv_bfloat16* hi;  // [T, 2 Fp]
  uint8_t* lo;        // [T, 2 Fp]
  __nv_bfloat16* a;   // [T, Fp]
};
static size_t carve_saved(void* p, const moe_ffn_config* c, Saved* s) {
  Carve cv(p);
  const size_t n = (size_t)c->T * pad64(c->F);
  s->hi = cv.take<__nv_bfloat16>(2 * n);
  s->lo = cv.take<uint8_t>(2 * n);
  s->a = cv.take<__nv_bfloat16>(n);
  return cv.used;
}

struct BwdWs {
  __nv_bfloat16* dgu;  // [T, 2 Fp]: dgate | dup
  float* part;
};
static size_t carve_bwd(void* ws, const moe_ffn_config* c, BwdWs* w) {
  Carve cv(ws);
  w->dgu = cv.take<__nv_bfloat16>((size_t)c->T * 2 * pad64(c->F));
  w->part = cv.take<float>(dense::PART_BYTES / sizeof(float));
  return cv.used;
}

// bf16 [outer, inner], boxes of 64 x box_outer.
static bool tmap(CUtensorMap* m, Mat a, long long inner, long long outer, int box_outer) {
  return moe_host::encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.p, inner, outer, (uint64_t)a.ld * 2, 64,
                                  box_outer);
}

static Params base_params(int M, int N, int KB, float* part, void* C, long long ldc) {
  Params p{};
  p.M = M;
  p.N = N;
  p.KB = KB;
  p.halves = 1;
  p.part = part;
  p.C = static_cast<__nv_bfloat16*>(C);
  p.ldc = ldc;
  p.status = moe_host::device_status_ptr();
  return p;
}

static int gateup(int T, int H, int F, Mat x, Mat Wg, Mat Wu, __nv_bfloat16* a, const Saved& s, float* part,
                  cudaStream_t st, bool dep) {
  Params p = base_params(T, F, cdiv(H, dense::BK), part, a, pad64(F));
  const dense::Plan c = dense::plan<dense::OP_GATEUP>(p);
  if (!tmap(&p.tmA, x, H, T, 128) || !tmap(&p.tmB0, Wg, H, F, c.b_box) || !tmap(&p.tmB1, Wu, H, F, c.b_box))
    return MOE_ERR_CUDA;
  p.save_hi = s.hi;
  p.save_lo = s.lo;
  p.ld2 = 2LL * pad64(F);
  p.up = pad64(F);
  return dense::launch<dense::OP_GATEUP>(p, c, st, dep);
}

static int down(int T, int H, int F, const __nv_bfloat16* a, Mat Wd, void* y, float* part, cudaStream_t st, bool dep) {
  const Mat am{a, pad64(F)};
  Params p = base_params(T, H, cdiv(F, dense::BK), part, y, H);
  const dense::Plan c = dense::plan<dense::OP_DOWN>(p);
  if (!tmap(&p.tmA, am, F, T, 128) || !tmap(&p.tmB0, Wd, F, H, c.b_box)) return MOE_ERR_CUDA;
  return dense::launch<dense::OP_DOWN>(p, c, st, dep);
}

static int dgrad_act(int T, int H, int F, Mat dY, Mat Wd, const Saved& s, __nv_bfloat16* dgu, float* part,
                     cudaStream_t st, bool dep) {
  Params p = base_params(T, F, cdiv(H, dense::BK), part, dgu, 0);
  const dense::Plan c = dense::plan<dense::OP_DGRAD_ACT>(p);
  if (!tmap(&p.tmA, dY, H, T, 128) || !tmap(&p.tmB0, Wd, F, H, 64)) return MOE_ERR_CUDA;
  p.save_hi = s.hi;
  p.save_lo = s.lo;
  p.ld2 = 2LL * pad64(F);
  p.up = pad64(F);
  return dense::launch<dense::OP_DGRAD_ACT>(p, c, st, dep);
}

static int dgrad_x(int T, int H, int F, const __nv_bfloat16* dgu, Mat Wg, Mat Wu, void* dX, float* part,
                   cudaStream_t st, bool dep) {
  const int kb = cdiv(F, dense::BK);
  const Mat dg{dgu, 2LL * pad64(F)}, du{dgu + pad64(F), 2LL * pad64(F)};
  Params p = base_params(T, H, 2 * kb, part, dX, H);
  const dense::Plan c = dense::plan<dense::OP_DGRAD_X>(p);
  p.kb_split = kb;
  if (!tmap(&p.tmA, dg, F, T, 128) || !tmap(&p.tmA2, du, F, T, 128) || !tmap(&p.tmB0, Wg, H, F, 64) ||
      !tmap(&p.tmB1, Wu, H, F, 64))
    return MOE_ERR_CUDA;
  return dense::launch<dense::OP_DGRAD_X>(p, c, st, dep);
}

// dW [M, N] = sum_t dO[t, :M]^T act[t, :N]; with dO2, a second [M, N] from it into dW2 in the same launch.
static int wgrad(int T, int M, int N, Mat dO, Mat dO2, Mat act, void* dW, void* dW2, float* part, cudaStream_t st,
                 bool dep) {
  Params p = base_params(M, N, cdiv(T, dense::BK), part, dW, N);
  p.halves = dO2.p ? 2 : 1;
  const dense::Plan c = dense::plan<dense::OP_WGRAD>(p);
  if (!tmap(&p.tmA, dO, M, T, 64) || !tmap(&p.tmB0, act, N, T, 64)) return MOE_ERR_CUDA;
  if (dO2.p) {
    if (!tmap(&p.tmA2, dO2, M, T, 64)) return MOE_ERR_CUDA;
    p.C2 = static_cast<__nv_bfloat16*>(dW2);
  }
  return dense::launch<dense::OP_WGRAD>(p, c, st, dep);
}

// One product of the streaming path: W1 for gate/up, scales for MXFP8; x has rows of ldx elements, out of ldo.
template <bool MX, bool GATEUP>
static int stream_gemm(int T, int N, int K, const void* W0, const void* W1, const uint8_t* sf0, const uint8_t* sf1,
                       Mat x, const uint8_t* x_sf, void* out, long long ldo, uint8_t* out_sf, const Saved& s,
                       cudaStream_t st, bool dep, const void* W_next = nullptr) {
  stream::Params p = stream::plan<MX, GATEUP>(T, N, K);
  if (GATEUP && !stream::plan_next<MX>(p, W_next)) return MOE_ERR_CUDA;
  if (!stream::encode_maps<MX>(&p.tmW0, &p.tmW0t, p, W0, N, p.r, K) ||
      (GATEUP && !stream::encode_maps<MX>(&p.tmW1, &p.tmW1t, p, W1, N, p.r, K)) ||
      !stream::encode_maps<MX>(&p.tmX, &p.tmXt, p, x.p, T, T, x.ld))
    return MOE_ERR_CUDA;
  p.sf0 = sf0;
  p.sf1 = sf1;
  p.x_sf = x_sf;
  p.out = out;
  p.ldo = ldo;
  p.out_sf = out_sf;
  p.save_hi = reinterpret_cast<uint16_t*>(s.hi);
  p.save_lo = s.lo;
  p.ld2 = 2LL * pad64(N);
  p.up = pad64(N);
  return stream::launch<MX, GATEUP>(p, st, dep);
}

// x [T, H] bf16 -> MXFP8 for the streaming path: a thread takes 8 elements, four lanes a 1x32 block. The kernel
// behind it may start at once (its weights do not depend on x).
__global__ void __launch_bounds__(256) quantize_kernel(const __nv_bfloat16* __restrict__ x, long long n8,
                                                       uint8_t* __restrict__ q, uint8_t* __restrict__ sf) {
  griddep_launch_dependents();
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const bool ok = i < n8;  // n8 % 4 == 0: the lanes of a block are all in or all out
  float v[8];
  unpack_bf16x8(ok ? *reinterpret_cast<const uint4*>(x + 8 * i) : make_uint4(0, 0, 0, 0), v);
  float am = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) am = fmaxf(am, fabsf(v[j]));
  am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
  am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
  const uint8_t sb = ggmx::mx_scale_byte(am);
  const float inv = ggmx::mx_inv_scale(sb);
  uint32_t w[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    w[k] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[4 * k] * inv, v[4 * k + 1] * inv), __NV_SATFINITE,
                                              __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[4 * k + 2] * inv, v[4 * k + 3] * inv), __NV_SATFINITE,
                                              __NV_E4M3)
               << 16;
  if (!ok) return;
  reinterpret_cast<uint2*>(q)[i] = make_uint2(w[0], w[1]);
  if ((threadIdx.x & 3) == 0) sf[i >> 2] = sb;
}

static int fwd_bf16(const moe_ffn_config* c, const void* x, const void* Wg, const void* Wu, const void* Wd, void* y,
                    __nv_bfloat16* a, const Saved& s, const FwdWs& w, cudaStream_t st) {
  const int T = c->T, H = c->H, F = c->F, Fp = pad64(F);
  if (streams(c)) {
    FFN_RC((stream_gemm<false, true>(T, F, H, Wg, Wu, nullptr, nullptr, Mat{x, H}, nullptr, a, Fp, nullptr, s, st,
                                     false, Wd)));
    return stream_gemm<false, false>(T, H, F, Wd, nullptr, nullptr, nullptr, Mat{a, Fp}, nullptr, y, H, nullptr,
                                     Saved{}, st, true);
  }
  FFN_RC(gateup(T, H, F, Mat{x, H}, Mat{Wg, H}, Mat{Wu, H}, a, s, w.part, st, false));
  return down(T, H, F, a, Mat{Wd, F}, y, w.part, st, true);
}

// One product in MXFP8: out [T, N] = x W0^T, or the activation of x W0^T and x W1^T with its scales.
template <int OP>
static int dense_mx(int T, int N, int K, const void* x, const uint8_t* x_sf, const void* W0, const uint8_t* sf0,
                    const void* W1, const uint8_t* sf1, void* out, uint8_t* out_sf, float* part, cudaStream_t st,
                    bool dep) {
  Params p = base_params(T, N, K / 128, part, out, N);
  const dense::Plan c = dense::plan<OP>(p);
  const auto map = [&](CUtensorMap* m, const void* a, int rows, int box) {
    return moe_host::encode_tmap_2d(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, K, rows, K, 128, box);
  };
  if (!map(&p.tmA, x, T, 128) || !map(&p.tmB0, W0, N, c.b_box) || (W1 && !map(&p.tmB1, W1, N, c.b_box)))
    return MOE_ERR_CUDA;
  p.sfa = x_sf;
  p.sfb0 = sf0;
  p.sfb1 = sf1;
  p.ld_sf = K / 32;
  p.sf16 = K % 512 == 0 && a16(x_sf) && a16(sf0) && a16(sf1);
  p.C_sf = out_sf;
  return dense::launch<OP>(p, c, st, dep);
}

static int fwd_mxfp8(const moe_ffn_config* c, const void* x, const uint8_t* x_sf, const void* Wg, const void* Wu,
                     const void* Wd, const uint8_t* Wg_sf, const uint8_t* Wu_sf, const uint8_t* Wd_sf, void* y,
                     const FwdWs& w, cudaStream_t st) {
  const int T = c->T, H = c->H, F = c->F;
  const bool quant = x_sf == nullptr;
  if (quant) {
    const long long n8 = (long long)T * H / 8;
    quantize_kernel<<<(unsigned)((n8 + 255) / 256), 256, 0, st>>>(static_cast<const __nv_bfloat16*>(x), n8, w.xq,
                                                                 w.xq_sf);
    MOE_CHECK_LAUNCH();
    x = w.xq;
    x_sf = w.xq_sf;
  }
  if (streams(c)) {
    FFN_RC((stream_gemm<true, true>(T, F, H, Wg, Wu, Wg_sf, Wu_sf, Mat{x, H}, x_sf, w.aq, F, w.aq_sf, Saved{}, st,
                                    quant, Wd)));
    return stream_gemm<true, false>(T, H, F, Wd, nullptr, Wd_sf, nullptr, Mat{w.aq, F}, w.aq_sf, y, H, nullptr,
                                    Saved{}, st, true);
  }
  FFN_RC((dense_mx<dense::OP_GATEUP_MX>(T, F, H, x, x_sf, Wg, Wg_sf, Wu, Wu_sf, w.aq, w.aq_sf, w.part, st, quant)));
  return dense_mx<dense::OP_DOWN_MX>(T, H, F, w.aq, w.aq_sf, Wd, Wd_sf, nullptr, nullptr, y, nullptr, w.part, st, true);
}

}  // namespace ffn

extern "C" size_t moe_ffn_workspace_size(const moe_ffn_config* cfg) {
  if (ffn::check_cfg(cfg)) return 0;
  ffn::FwdWs w;
  return ffn::carve_fwd(nullptr, cfg, &w);
}

extern "C" size_t moe_ffn_saved_size(const moe_ffn_config* cfg) {
  if (ffn::check_cfg(cfg) || cfg->dtype != MOE_DT_BF16) return 0;
  ffn::Saved s;
  return ffn::carve_saved(nullptr, cfg, &s);
}

extern "C" size_t moe_ffn_bwd_workspace_size(const moe_ffn_config* cfg) {
  if (ffn::check_cfg(cfg) || cfg->dtype != MOE_DT_BF16) return 0;
  ffn::BwdWs w;
  return ffn::carve_bwd(nullptr, cfg, &w);
}

extern "C" int moe_ffn_fwd(const moe_ffn_config* cfg, const void* x, const uint8_t* x_sf, const void* W_g,
                           const void* W_u, const void* W_d, const uint8_t* W_g_sf, const uint8_t* W_u_sf,
                           const uint8_t* W_d_sf, void* y, void* saved, void* ws, size_t ws_bytes, void* stream) {
  using namespace ffn;
  FFN_RC(check_cfg(cfg));
  if (!x || !W_g || !W_u || !W_d || !y) return MOE_ERR_INVALID_ARG;
  const bool mx = cfg->dtype == MOE_DT_MXFP8;
  if (mx ? (!W_g_sf || !W_u_sf || !W_d_sf) : (x_sf || W_g_sf || W_u_sf || W_d_sf)) return MOE_ERR_INVALID_ARG;
  if ((cfg->save_for_bwd != 0) != (saved != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!a16(x) || !a16(W_g) || !a16(W_u) || !a16(W_d) || !a16(y) || !a16(saved) || !a16(ws) || !a4(x_sf) ||
      !a4(W_g_sf) || !a4(W_u_sf) || !a4(W_d_sf))
    return MOE_ERR_ALIGNMENT;
  FwdWs w;
  const size_t need = carve_fwd(nullptr, cfg, &w);
  if (need > 0 && (!ws || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  carve_fwd(ws, cfg, &w);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (mx) return fwd_mxfp8(cfg, x, x_sf, W_g, W_u, W_d, W_g_sf, W_u_sf, W_d_sf, y, w, st);
  Saved s{};
  if (saved) carve_saved(saved, cfg, &s);
  return fwd_bf16(cfg, x, W_g, W_u, W_d, y, saved ? s.a : w.a, s, w, st);
}

extern "C" int moe_ffn_bwd(const moe_ffn_config* cfg, const void* dY, const void* x, const void* W_g, const void* W_u,
                           const void* W_d, const void* saved, void* dX, void* dW_g, void* dW_u, void* dW_d, void* ws,
                           size_t ws_bytes, void* stream) {
  using namespace ffn;
  FFN_RC(check_cfg(cfg));
  if (cfg->dtype != MOE_DT_BF16) return MOE_ERR_UNSUPPORTED;
  if (!cfg->save_for_bwd || !dY || !W_d || !saved) return MOE_ERR_INVALID_ARG;
  if ((dW_g == nullptr) != (dW_u == nullptr) || (!dX && !dW_g && !dW_d)) return MOE_ERR_INVALID_ARG;
  if ((dX && (!W_g || !W_u)) || (dW_g && !x)) return MOE_ERR_INVALID_ARG;
  if (!a16(dY) || !a16(x) || !a16(W_g) || !a16(W_u) || !a16(W_d) || !a16(saved) || !a16(dX) || !a16(dW_g) ||
      !a16(dW_u) || !a16(dW_d) || !a16(ws))
    return MOE_ERR_ALIGNMENT;
  BwdWs w;
  if (!ws || ws_bytes < carve_bwd(nullptr, cfg, &w)) return MOE_ERR_WORKSPACE;
  carve_bwd(ws, cfg, &w);
  Saved s;
  carve_saved(const_cast<void*>(saved), cfg, &s);
  const int T = cfg->T, H = cfg->H, F = cfg->F;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int Fp = pad64(F);
  const Mat mdy{dY, H}, mx{x, H}, mg{W_g, H}, mu{W_u, H}, md{W_d, F};
  bool dep = false;
  if (dX || dW_g) {
    FFN_RC(dgrad_act(T, H, F, mdy, md, s, w.dgu, w.part, st, dep));
    dep = true;
  }
  if (dW_d) {
    FFN_RC(wgrad(T, H, F, mdy, Mat{}, Mat{s.a, Fp}, dW_d, nullptr, w.part, st, dep));
    dep = true;
  }
  if (dX) FFN_RC(dgrad_x(T, H, F, w.dgu, mg, mu, dX, w.part, st, dep));
  if (dW_g)
    FFN_RC(wgrad(T, F, H, Mat{w.dgu, 2LL * Fp}, Mat{w.dgu + Fp, 2LL * Fp}, mx, dW_g, dW_u, w.part, st, true));
  return MOE_OK;
}
