// Forms of the dense feed-forward GEMM that plan_for() gives, on 148 SMs. Two lines per product of a size:
//   product:CTAs per tile x columns:split T H F   split  whole | cut (a piece per CTA, added by one thread) |
//                                                        many (the same, by four) | line
//   product:order T H F                           order  m or n (first), with g in groups of panels
// dense_plan bf16|mx PAIRS list T H F ...      the products of these sizes
// dense_plan bf16|mx PAIRS search COUNT SEED   each form once, at the size of least work found
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <random>
#include <string>

#include "../mixture_experts_layer_aux_b200/csrc/dense.cuh"
#include "../mixture_experts_layer_aux_b200/csrc/stream.cuh"

namespace moe_host {
int num_sms() { return 148; }
int* device_status_ptr() { return nullptr; }
bool encode_tmap_3d(CUtensorMap*, CUtensorMapDataType, const void*, uint64_t, uint64_t, uint64_t, uint64_t, uint64_t,
                    uint32_t, uint32_t, uint32_t) {
  return false;
}
}  // namespace moe_host

using namespace dense;
static int g_pairs;
struct Size {
  int T, H, F;
  double work() const { return (double)T * H * F; }
};
static std::map<std::string, Size> g_best;
static bool g_list;

template <int OP>
static void product(const char* name, const Size& z, int M, int N, int KB, int halves = 1) {
  Params p{};
  p.M = M;
  p.N = N;
  p.KB = KB;
  p.halves = halves;
  const Plan c = plan_for<OP>(p, 148, g_pairs);
  // the pieces of a tile are one per CTA where its place on the line is a whole number of them
  const bool line = p.sk_tiles && p.sk_kb % p.sk_per != 0;
  const char* split = !p.sk_tiles ? "whole" : line ? "line" : KB > MANY_PIECES * p.sk_per ? "many" : "cut";
  const int fast = p.n_fast ? p.tiles_n : p.tiles_m;
  char form[96], order[96];
  std::snprintf(form, sizeof form, "%s:%dx%d:%s", name, c.cg, c.bn, split);
  std::snprintf(order, sizeof order, "%s:%s%s", name, p.n_fast ? "n" : "m", p.group < fast ? "g" : "");
  for (const char* key : {form, order}) {
    if (g_list) std::printf("%s %d %d %d\n", key, z.T, z.H, z.F);
    const auto at = g_best.find(key);
    if (at == g_best.end() || z.work() < at->second.work()) g_best[key] = z;
  }
}

static void products(const Size& z, bool mx) {
  const auto kb = [](int k) { return (k + 63) / 64; };
  if (mx) {
    if (z.T <= stream::MAX_T_MX) return;
    product<OP_GATEUP_MX>("gateup_mx", z, z.T, z.F, z.H / 128);
    product<OP_DOWN_MX>("down_mx", z, z.T, z.H, z.F / 128);
    return;
  }
  if (z.T > stream::MAX_T) {
    product<OP_GATEUP>("gateup", z, z.T, z.F, kb(z.H));
    product<OP_DOWN>("down", z, z.T, z.H, kb(z.F));
  }
  product<OP_DGRAD_ACT>("dgrad_act", z, z.T, z.F, kb(z.H));
  product<OP_DGRAD_X>("dgrad_x", z, z.T, z.H, 2 * kb(z.F));
  product<OP_WGRAD>("wgrad", z, z.H, z.F, kb(z.T));
  product<OP_WGRAD>("wgrad2", z, z.F, z.H, kb(z.T), 2);
}

int main(int argc, char** argv) {
  if (argc < 5) return 1;
  const bool mx = !std::strcmp(argv[1], "mx");
  g_pairs = std::atoi(argv[2]);
  g_list = !std::strcmp(argv[3], "list");
  if (g_list) {
    for (int i = 4; i + 2 < argc; i += 3)
      products({std::atoi(argv[i]), std::atoi(argv[i + 1]), std::atoi(argv[i + 2])}, mx);
    return 0;
  }
  std::mt19937 rng(std::atoi(argv[5]));
  const auto log_between = [&](double lo, double hi) {
    return lo * std::pow(hi / lo, rng() / 4294967296.0);
  };
  for (int i = 0; i < std::atoi(argv[4]); ++i) {
    Size z;
    z.T = (int)log_between(1, 8192);
    z.H = mx ? 256 * (int)log_between(1, 40) : 8 * (int)log_between(8, 1024);
    z.F = mx ? 128 * (int)log_between(1, 128) : 8 * (int)log_between(8, 2048);
    products(z, mx);
  }
  for (const auto& b : g_best)
    std::printf("%s %d %d %d\n", b.first.c_str(), b.second.T, b.second.H, b.second.F);
}
