// Checks of the record of prepared workspaces (csrc/gla_prepared.h) on made-up
// addresses; returns the number of those that fail.
#include <stdio.h>

#include "gla_prepared.h"

static int failed = 0;
#define EXPECT(x) \
  if (!(x)) ++failed, printf("line %d: %s\n", __LINE__, #x)

int main() {
  const size_t ctrl = 65536, MiB = 1 << 20;
  auto at = [](size_t a) { return reinterpret_cast<const void*>(a); };
  gla::Prepared p(ctrl);
  const size_t ws = 16 * MiB;
  EXPECT(!p.contains(at(ws)) && !p.control_words_in(at(ws), MiB));
  p.add(at(ws), 4 * MiB);
  EXPECT(p.contains(at(ws)) && !p.contains(at(ws + 256)));
  EXPECT(p.control_words_in(at(ws), MiB));
  EXPECT(p.control_words_in(at(ws + 256), MiB));           // starts inside the control words
  EXPECT(p.control_words_in(at(ws + ctrl - 256), 256));    // their last bytes
  EXPECT(p.control_words_in(at(ws - MiB), 2 * MiB));       // runs over them from before
  EXPECT(p.control_words_in(at(ws - MiB), MiB + 1));
  EXPECT(!p.control_words_in(at(ws - MiB), MiB));          // ends where they start
  EXPECT(!p.control_words_in(at(ws + ctrl), MiB));         // behind them, in the same buffer
  p.add(at(ws + 8 * MiB), ctrl);
  EXPECT(p.control_words_in(at(ws + 8 * MiB + 256), 256) && p.control_words_in(at(ws + 256), 256));
  p.remove(at(ws));
  EXPECT(!p.contains(at(ws)) && !p.control_words_in(at(ws), MiB));
  EXPECT(p.control_words_in(at(ws), 9 * MiB));             // the other one
  p.remove(at(ws));                                        // not there: nothing happens
  p.remove(at(ws + 8 * MiB));
  EXPECT(!p.control_words_in(at(0), 64 * MiB));
  return failed;
}
