// tw_rows_q8.cu -- the rows kernel's instantiations with 8-bit outputs.
#include "tw_rows.cuh"

namespace tw {

void* rows_q8_entry(int dtype, int nv, int unit, int mode) {
    return rows_entry<true>(dtype, nv, unit, mode);
}

void* rows2_q8_entry(int dtype, int nv, int unit) { return rows2_entry<true>(dtype, nv, unit); }

}  // namespace tw
