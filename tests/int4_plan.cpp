// Prints the kernel and the split of a 4-bit product for "gate_up group routed_rows experts blocks
// outputs columns chunks" lines.
#include <cstdio>

#include "int4_plan.h"

int main() {
  using namespace moe;
  const char* names[] = {"rows16", "rows32", "tiles"};
  int up, group, rows, experts, blocks, outputs, columns;
  long long chunks;
  while (std::scanf("%d %d %d %d %d %d %d %lld", &up, &group, &rows, &experts, &blocks, &outputs, &columns, &chunks) == 8)
    std::printf("%s %d\n", names[static_cast<int>(int4_kernel(up != 0, group, rows, experts))],
                int4_split(blocks, outputs, columns, chunks));
  return 0;
}
