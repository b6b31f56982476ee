// The rule of fa_rows.h for rows of a batch behind a C interface, for the tests.
#include "../../flash_attention_gb300/csrc/fa_rows.h"

extern "C" int grids_meet(const int64_t* na, const int64_t* sa, const int64_t* nb, const int64_t* sb,
                          int64_t offset, int64_t d) {
  fa::RowBox a, b;
  for (int k = 0; k < 3; ++k) a.n[k] = na[k], a.st[k] = sa[k], b.n[k] = nb[k], b.st[k] = sb[k];
  return fa::boxes_meet(a, b, offset, d);
}
