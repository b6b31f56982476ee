// The row-overlap rules of fa_rows.h behind a C interface, for the tests.
#include "../../flash_attention_gb300/csrc/fa_rows.h"

extern "C" int rows_are_apart(int64_t heads, int64_t rows, int64_t d, int64_t k_h, int64_t k_r,
                              int64_t v_h, int64_t v_r, int64_t offset) {
  return fa::rows_apart({heads, rows, k_h, k_r}, {heads, rows, v_h, v_r}, offset, d);
}
