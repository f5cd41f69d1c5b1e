// Prints what the launch rules of csrc/block_launch.h choose, one line per query of the command
// line's (a name and its numbers; bf16 is 1, fp32 0). Host only; built and run by
// tests/test_block_launch_rules.py.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "block_launch.h"

int main(int argc, char** argv) {
  int i = 1;
  auto num = [&] { return i < argc ? strtoll(argv[i++], nullptr, 10) : -1; };
  while (i < argc) {
    const char* name = argv[i++];
    if (!strcmp(name, "conv_fwd")) {  // batch dim seqlen io
      const int64_t b = num(), d = num(), L = num();
      const ssm::Io io = num() ? ssm::Io::BF16 : ssm::Io::F32;
      printf("%d\n", ssm::conv_fwd_wave_tiles(b, d, L, io));
    } else if (!strcmp(name, "conv_step")) {  // batch dim io
      const int64_t b = num(), d = num();
      printf("%d\n", ssm::conv_step_rows(b, d, num() ? ssm::Io::BF16 : ssm::Io::F32));
    } else if (!strcmp(name, "state_step")) {  // batch dim dstate: channels past_caches
      const int64_t b = num(), d = num();
      const ssm::StepForm f = ssm::step_form(b, d, num());
      printf("%d %d\n", f.channels, int(f.past_caches));
    } else if (!strcmp(name, "norm_fwd") || !strcmp(name, "norm_bwd")) {
      // batch dim groups seqlen io all_channel dword_rows: steps lanes_log2 waves split
      const int64_t b = num(), d = num(), g = num(), L = num();
      const ssm::Io io = num() ? ssm::Io::BF16 : ssm::Io::F32;
      const bool chan = num() != 0, dword = num() != 0;
      const ssm::NormShape s = strcmp(name, "norm_fwd") ? ssm::norm_bwd_shape(b, d, g, L, io, {chan, dword})
                                                        : ssm::norm_fwd_shape(b, d, g, L, io, {chan, dword});
      printf("%d %d %d %d\n", s.steps, s.lanes_log2, s.waves, int(s.split));
    } else {
      return 1;
    }
  }
  return 0;
}
