#include "ce_rows_kernel.cuh"

namespace gbce {
const void* rows_kernel_bf16(int op, bool ent, int nt) { return rows_kernel_of<__nv_bfloat16>(op, ent, nt); }
}  // namespace gbce
