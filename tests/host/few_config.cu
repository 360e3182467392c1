// Host program: the pipeline constants of each few-token kernel, one line per
// instantiation, for the protocol model.
#include <cstdio>

#include "few.cuh"

template <int MODE, int NT, bool kBf16>
void line(const char* name) {
  using C = fgfp8::FewCfg<MODE, NT>;
  std::printf("%s stages=%d slots=%d buffers=%d epi_warps=%d groups=%d token_warps=%d mma_warps=%d red_tokens=%d max_s=%d "
              "copies=%d ring=%d\n",
              name, C::kStages, C::kScSlots, C::kNumBuf, C::kEpiWarps, C::kGroups, C::kTokWarps, C::kMmaWarps, C::kRedTok,
              C::kMaxS, kBf16 ? 0 : 1, MODE == fgfp8::kFewDown && C::kGroups > 1 ? 1 : 0);
}

int main() {
  line<fgfp8::kFewGateUp, 16, true>("gate_up_16");
  line<fgfp8::kFewGateUp, 64, false>("gate_up_64");
  line<fgfp8::kFewDown, 16, false>("down_16");
  line<fgfp8::kFewDown, 64, false>("down_64");
  line<fgfp8::kFewLinear, 16, true>("linear_16_bf16");
  line<fgfp8::kFewLinear, 16, false>("linear_16");
  line<fgfp8::kFewLinear, 64, false>("linear_64");
}
