#include "ce_rows_kernel.cuh"

namespace gbce {
const void* rows_kernel_f32(int op, bool ent, int nt) { return rows_kernel_of<float>(op, ent, nt); }
}  // namespace gbce
