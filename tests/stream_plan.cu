// Prints what the gate/up kernel of the streaming path asks into L2 for the down kernel, as `plan_next` lays it out and
// the kernel walks it. Arguments: T H F triples. Per triple one line
//   T H F : cs KS stages s r tiles bytes-of-a-stage budget : rank:from-to ...
// with the stages that each CTA of tile 0 has asked for (they are the same for every tile).
#include <cstdio>
#include <cstdlib>

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

int main(int argc, char** argv) {
  const bool mx = argc > 1 && argv[1][0] == 'm';
  for (int i = 2; i + 2 < argc; i += 3) {
    const int T = atoi(argv[i]), H = atoi(argv[i + 1]), F = atoi(argv[i + 2]);
    if (mx) show<true>(T, H, F);
    else show<false>(T, H, F);
  }
}
