// The kernel choice of the expert operators (csrc/expert_forms.hpp, host code) for
// the sizes on standard input, for tests/test_expert_forms.py.  A line in, a line out:
//   p TYPE M E n k TRANSPOSE SWIGLU   ->  form (TYPE 0 float32, 1 bf16, 2 int8)
//   w BF16 M E n k                    ->  tile part slots
#include <cstdio>

#include "hip/hip_runtime.h"
#include "expert_forms.hpp"

int main() {
  char kind;
  int t, M, E, n, k;
  while (std::scanf(" %c %d %d %d %d %d", &kind, &t, &M, &E, &n, &k) == 6) {
    if (kind == 'p') {
      omni::ExpertMatmulArgs a = {};
      a.type = t;
      a.M = M, a.E = E, a.n = n, a.k = k;
      if (std::scanf("%d %d", &a.transpose, &a.swiglu) != 2) return 2;
      std::printf("%d\n", omni::pick_form(a));
    } else {
      const omni::WgradPlan p = omni::plan_wgrad(t, M, E, n, k);
      std::printf("%d %d %d\n", p.tile, p.part, p.slots);
    }
  }
  return 0;
}
