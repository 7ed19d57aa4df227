// Host check of the batch calls' rule on shared memory: prints one digit per case.
#include <cstdio>

#include "wf_batch.h"

int main() {
  static char m[64];
  using wf::Span;
  const struct {
    Span a, b;
    bool want;
  } cases[] = {
      {{m, 16}, {m, 16}, true},           {{m, 16}, {m + 16, 16}, false},    {{m, 16}, {m + 15, 16}, true},
      {{m + 8, 16}, {m, 9}, true},        {{m + 8, 16}, {m, 8}, false},      {{m, 64}, {m + 20, 4}, true},
      {{m + 20, 4}, {m, 64}, true},       {{m, 0}, {m, 16}, false},          {{m + 4, 0}, {m, 16}, false},
      {{nullptr, 16}, {m, 16}, false},    {{nullptr, 16}, {nullptr, 16}, false},
      {{m, 1}, {m, 1}, true},             {{m, ~size_t(0)}, {m + 63, 1}, true},
  };
  int bad = 0;
  for (const auto& c : cases) {
    bad += wf::overlap(c.a, c.b) != c.want;
    bad += wf::overlap(c.b, c.a) != c.want;
  }
  // outputs against inputs and against one another; inputs may share memory
  const Span in[] = {{m, 16}, {m + 8, 16}};
  const Span clear[] = {{m + 24, 8}, {m + 32, 8}}, on_input[] = {{m + 32, 8}, {m + 23, 8}}, twice[] = {{m + 24, 9}, {m + 32, 8}};
  bad += wf::written_over(clear, in) || !wf::written_over(on_input, in) || !wf::written_over(twice, in);
  std::printf("%d wrong\n", bad);
  return bad != 0;
}
