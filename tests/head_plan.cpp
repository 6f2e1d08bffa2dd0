// Prints what the head's loss does for sizes given as "rows cols vocab" lines: one JSON line each.
#include <cstdio>

#include "head_plan.h"

int main() {
  using namespace moe;
  const char* names[] = {"rows32", "rows64", "mid", "wide"};
  long long rows;
  int cols, vocab;
  while (std::scanf("%lld %d %d", &rows, &cols, &vocab) == 3) {
    const Plan q = plan(static_cast<int>(rows), cols, vocab);
    std::printf("{\"forward\": \"%s\", \"dx\": \"%s\", \"parts\": %d, \"sums\": %s, \"bytes\": %zu, \"bound\": %zu, \"pieces\": [",
                names[tile_of_logits(rows, vocab, cols)], names[q.tile], q.parts, q.sums ? "true" : "false", q.bytes,
                workspace_bound(rows, cols, vocab));
    for (int v0 = 0; v0 < vocab; v0 += q.piece) {
      const int width = piece_width(q, v0, vocab);
      std::printf("%s{\"width\": %d, \"probs\": \"%s\", \"dw\": \"%s\", \"parts\": %d}", v0 ? ", " : "", width,
                  names[tile_of_logits(rows, width, cols)], names[tile_of_dw(q, width, cols)], parts_of_dx(q, width));
    }
    std::printf("]}\n");
  }
  return 0;
}
