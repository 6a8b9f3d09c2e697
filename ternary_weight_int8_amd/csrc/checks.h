// checks.h -- host checks of the calls' buffers.
#ifndef TERNARY_CHECKS_H
#define TERNARY_CHECKS_H

#include <stdint.h>

namespace {

bool overlap(const void *a, int64_t an, const void *b, int64_t bn) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && an > 0 && bn > 0 && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}
bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Buf {
  const void *p;
  int64_t bytes;
};
// whether outs[i] overlaps an input (equal pointers allowed where `same` names
// that input for it) or a later output; NULL buffers overlap nothing
template <int NO, int NI>
bool alias(const Buf (&outs)[NO], const Buf (&ins)[NI], const void *const (&same)[NO][2]) {
  for (int i = 0; i < NO; ++i) {
    for (int j = 0; j < NI; ++j)
      if (overlap(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes) &&
          !(outs[i].p == ins[j].p && outs[i].bytes == ins[j].bytes &&
            (ins[j].p == same[i][0] || ins[j].p == same[i][1])))
        return true;
    for (int j = i + 1; j < NO; ++j)
      if (overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
  }
  return false;
}

bool workspace_ok(const void *ws, int64_t bytes, int64_t need) {
  return need == 0 || (ws && bytes >= need && aligned(ws, 16));
}

}  // namespace

#endif  // TERNARY_CHECKS_H
