// Prints csrc/launch_rule.h's answers for lines of arguments read from stdin: "c M N TN" the
// column tiles of a launch, "k M N E f4 wide cus" the linear layer's kernel (0: 16 rows, 1:
// 128-row tiles, 2: pipeline), "w M N E cus" the waves of its 16-row kernel.
#include "launch_rule.h"

#include <cstdio>

int main() {
  long long M, N, E, cus;
  int tn, f4, wide;
  char what;
  while (std::scanf(" %c", &what) == 1) {
    long long v = -1;
    if (what == 'c' && std::scanf("%lld %lld %d", &M, &N, &tn) == 3) v = mx::column_tiles(M, N, tn);
    else if (what == 'k' && std::scanf("%lld %lld %lld %d %d %lld", &M, &N, &E, &f4, &wide, &cus) == 6)
      v = (int)mx::linear_kernel(M, N, E, f4 != 0, wide != 0, cus);
    else if (what == 'w' && std::scanf("%lld %lld %lld %lld", &M, &N, &E, &cus) == 4)
      v = mx::rows16_waves(M, N, E, cus);
    std::printf("%lld\n", v);
  }
  return 0;
}
