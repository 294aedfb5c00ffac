// Runs the prompt attention's join on parts that the host makes: a unit of 256 rows cut between
// `spans` CTAs, whose part i holds m = 0, l = 1 and O = i + 1 in every row.  `gave_up`: the CTA
// that says a wait of its ran out (-1: none).
#include "../../paged_mla_latent_gb300/csrc/mla_prompt_attention.cu"

#include <vector>

namespace pmla {
void* tensor_map_encoder() { return nullptr; }
}  // namespace pmla

// o (256, 64) bf16 bits and lse (256) on the host: filled in with what the join leaves, over the
// caller's own contents.  Returns the parts that the unit has, or minus a CUDA error.
extern "C" int prompt_join_probe(int spans, int gave_up, uint16_t* o, float* lse) {
  using namespace pmla;
  constexpr int DV = 64, kPart = 2 * kRows * (DV + 2);
  const int64_t tiles = 16 * spans, weight = kUnitCost + tiles * kKeys;
  const int64_t span = (weight + spans - 1) / spans;
  Piece unit = {0, 256, static_cast<int>(tiles) * kKeys - 256, 0, 0, 0, 0, 1};
  std::vector<Cut> cuts(spans);
  std::vector<float> parts(static_cast<size_t>(2) * spans * kPart, 1e30f);     // stale
  int n = 0, t = 0;
  for (int i = 0; i < spans; ++i) {
    cuts[i] = {};
    cuts[i].gave_up = i == gave_up;
    const int e = i + 1 == spans ? static_cast<int>(tiles)
                                 : cut_at(0, weight, static_cast<int>(tiles), (i + 1) * span, true);
    if (i == 0) {
      if (e <= 0 || e >= tiles) return -1000;
      unit.j1 = e;
      cuts[0].unit = unit;
      cuts[0].tiles = static_cast<int>(tiles);
      cuts[0].weight = weight;
      cuts[0].span = span;
    }
    if (e <= t) continue;
    t = e;
    float* at = parts.data() + (2 * i + (i == 0 ? 1 : 0)) * static_cast<size_t>(kPart);
    for (int r = 0; r < 2 * kRows; ++r) {
      at[r] = 0.f;
      at[2 * kRows + r] = 1.f;
      for (int d = 0; d < DV; ++d) at[4 * kRows + r * DV + d] = static_cast<float>(n + 1);
    }
    ++n;
  }
  PromptParams p = {};
  p.B = p.Hq = p.Hk = p.G = 1;
  p.tok_tile = kRows;
  p.o_tok = p.o_head = DV;
  void* mem[4] = {};
  const size_t bytes[4] = {cuts.size() * sizeof(Cut), parts.size() * 4, 256 * DV * 2, 256 * 4};
  const void* from[4] = {cuts.data(), parts.data(), o, lse};
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 4 && e == cudaSuccess; ++i) {
    e = cudaMalloc(&mem[i], bytes[i]);
    if (e == cudaSuccess) e = cudaMemcpy(mem[i], from[i], bytes[i], cudaMemcpyHostToDevice);
  }
  if (e == cudaSuccess) {
    p.cuts = static_cast<Cut*>(mem[0]);
    p.parts = static_cast<float*>(mem[1]);
    p.o = static_cast<uint16_t*>(mem[2]);
    p.lse = static_cast<float*>(mem[3]);
    prompt_join_kernel<DV><<<dim3(spans - 1, 8), 256>>>(p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) e = cudaMemcpy(o, mem[2], bytes[2], cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemcpy(lse, mem[3], bytes[3], cudaMemcpyDeviceToHost);
  for (void* m : mem) cudaFree(m);
  return e == cudaSuccess ? n : -static_cast<int>(e);
}
