// Plans of the streaming kernels on 148 SMs.
// stream_plan bf16|mx T H F ...          what the gate/up kernel asks into L2 for the down kernel, as plan_next() lays
//   it out and the kernel walks it; per size one line
//     T H F : cs KS stages s r tiles bytes-of-a-stage budget : rank:from-to ...
//   with the stages for each CTA of tile 0 (they are the same for every tile)
// stream_plan bf16|mx list T H F ...     forms of both products of these sizes, a line "form T H F" each
// stream_plan bf16|mx search COUNT SEED  each form once, at the size of least work found
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <random>
#include <string>

#include "../mixture_experts_layer_aux_b200/csrc/stream.cuh"

namespace moe_host {
int num_sms() { return 148; }
int* device_status_ptr() { return nullptr; }
bool encode_tmap_2d(CUtensorMap*, CUtensorMapDataType, const void*, uint64_t, uint64_t, uint64_t, uint32_t, uint32_t) {
  return true;
}
bool encode_tmap_3d(CUtensorMap*, CUtensorMapDataType, const void*, uint64_t, uint64_t, uint64_t, uint64_t, uint64_t,
                    uint32_t, uint32_t, uint32_t) {
  return true;
}
}  // namespace moe_host

template <bool MX>
static void show(int T, int H, int F) {
  using namespace stream;
  Params p = plan<MX, true>(T, F, H);
  const Params d = plan<MX, false>(T, H, F);
  if (!plan_next<MX>(p, nullptr)) exit(1);
  std::printf("%d %d %d : %d %d %d %d %d %d %d %lld :", T, H, F, d.cs, d.KS, d.stages, d.s, d.r, d.tiles,
              d.s * d.r * ROW_BYTES, NEXT_BYTES);
  for (int j = 0; j < p.next_tiles * p.next_cs && j < p.next_cs; ++j) {
    int from, to;
    next_stages(p, j, from, to);
    if (from >= to) from = to = -1;
    std::printf(" %d:%d-%d", j, from, to);
  }
  std::printf("\n");
}

struct Size {
  int T, H, F;
  double work() const { return (double)T * H * F; }
};

// What a plan can choose: CTAs per tile, gate and up in one operand, several K blocks per stage and whether the last
// stage has all of them, a tail of K, maps cut along K, rounds of tiles (1, 2, more), accumulators.
template <bool MX, bool GATEUP>
static std::string form(int T, int N, int K) {
  const stream::Params p = stream::plan<MX, GATEUP>(T, N, K);
  const int rounds = (p.tiles + 147) / 148;
  char b[128];
  std::snprintf(b, sizeof b, "%s:%d:%s:%s:%s:%s:%d:%d", GATEUP ? "gateup" : "down", p.cs, p.merged ? "merged" : "-",
                p.s == 1 ? "-" : p.KB % p.s ? "ragged" : "stacked", p.tail ? "tail" : "-", p.z ? "z" : "-",
                rounds < 3 ? rounds : 3, p.acc_bufs);
  return b;
}

static std::map<std::string, Size> g_best;
static void forms(const Size& z, bool mx, bool list) {
  const std::string keys[2] = {mx ? form<true, true>(z.T, z.F, z.H) : form<false, true>(z.T, z.F, z.H),
                               mx ? form<true, false>(z.T, z.H, z.F) : form<false, false>(z.T, z.H, z.F)};
  for (const std::string& k : keys) {
    if (list) std::printf("%s %d %d %d\n", k.c_str(), z.T, z.H, z.F);
    const auto at = g_best.find(k);
    if (at == g_best.end() || z.work() < at->second.work()) g_best[k] = z;
  }
}

int main(int argc, char** argv) {
  if (argc < 3) return 1;
  const bool mx = argv[1][0] == 'm', list = !std::strcmp(argv[2], "list");
  const int most = mx ? stream::MAX_T_MX : stream::MAX_T;
  if (!std::strcmp(argv[2], "search")) {
    std::mt19937 rng(std::atoi(argv[4]));
    const auto log_between = [&](double lo, double hi) { return lo * std::pow(hi / lo, rng() / 4294967296.0); };
    for (int i = 0; i < std::atoi(argv[3]); ++i) {
      Size z;
      z.T = 1 + (int)(rng() % most);
      z.H = mx ? 256 * (int)log_between(1, 100) : 8 * (int)log_between(1, 3000);
      z.F = mx ? 128 * (int)log_between(1, 200) : 8 * (int)log_between(1, 3000);
      forms(z, mx, false);
    }
    for (const auto& b : g_best)
      std::printf("%s %d %d %d\n", b.first.c_str(), b.second.T, b.second.H, b.second.F);
    return 0;
  }
  for (int i = list ? 3 : 2; i + 2 < argc; i += 3) {
    const int T = std::atoi(argv[i]), H = std::atoi(argv[i + 1]), F = std::atoi(argv[i + 2]);
    if (list) {
      if (T <= most) forms({T, H, F}, mx, true);
    } else if (mx) {
      show<true>(T, H, F);
    } else {
      show<false>(T, H, F);
    }
  }
}
