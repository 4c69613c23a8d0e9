// The kernel choice of the 4-bit products (csrc/expert_forms.hpp, host code) for the
// sizes on standard input, for tests/test_microscale_forms.py.  A line in, a line out:
//   M E n k SWIGLU   ->  form tiles workgroups
#include <cstdio>

#include "hip/hip_runtime.h"
#include "expert_forms.hpp"

int main() {
  omni::ExpertMatmulArgs a = {};
  while (std::scanf("%d %d %d %d %d", &a.M, &a.E, &a.n, &a.k, &a.swiglu) == 5) {
    const omni::MxForm f = omni::pick_mx_form(a);
    std::printf("%d %lld %lld\n", f, omni::mx_tiles(a, f), omni::mx_blocks(a, f));
  }
  return 0;
}
