// Which copies into a ring of stages may still be under way when their
// reader has given up.  Plain C++, so that it is tested on the host.
#pragma once

namespace w8 {

// Fillings of a ring of `ring` stages are numbered from 0; number e goes to stage e % ring.  A
// copier does every `step`-th of them and would do `next` next; where step is 2, the
// fillings between are another copier's, which would do `other` next (ring is
// odd then, so that the two take turns at each stage).  Of the copier's last fillings the j-th
// from the end, j = 1 .. ring: its number, or -1 where there is none, or where the stage has
// been filled again since, which is done only after a reader has seen it full.
constexpr int unread_filling(int next, int other, int step, int ring, int j) {
  const int e = next - step * j;
  if (e < 0) return -1;
  return step == 2 && e + ring < other ? -1 : e;
}

}  // namespace w8
