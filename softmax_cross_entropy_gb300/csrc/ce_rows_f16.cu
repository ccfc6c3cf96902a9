#include "ce_rows_kernel.cuh"

namespace gbce {
const void* rows_kernel_f16(int op, bool ent, int nt) { return rows_kernel_of<__half>(op, ent, nt); }
}  // namespace gbce
