// Reads pairs "M N" and prints the number of the kernel that mx_linear takes for each.
#include <inttypes.h>
#include <stdio.h>

#include "linear_plan.h"

int main() {
  int64_t m, n;
  while (scanf("%" SCNd64 " %" SCNd64, &m, &n) == 2) printf("%d\n", (int)mxk::linear_kernel(m, n));
  return 0;
}
