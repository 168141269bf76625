// Prints csrc/launch_rule.h's answers for lines of arguments read from stdin.
#include "launch_rule.h"

#include <cstdio>

int main() {
  long long M, N;
  int tn;
  while (std::scanf("%lld %lld %d", &M, &N, &tn) == 3) std::printf("%lld\n", (long long)mx::column_tiles(M, N, tn));
  return 0;
}
