// kvc_rows_inst.cu -- the tensor-core prompt and tree attention for one 16-bit
// element type and head width, selected at compile time by KVC_INST_TYPE
// (0 bf16, 1 fp16) and KVC_INST_D (64 or 128).
#include "kvc_rows_tc.cuh"

#if KVC_INST_TYPE == 0
#define KVC_ELEM __nv_bfloat16
#define KVC_TAG bf16
#else
#define KVC_ELEM __half
#define KVC_TAG f16
#endif

#define KVC_RCAT2(a, b) rows_kernel_##a##_##b
#define KVC_RCAT(a, b) KVC_RCAT2(a, b)

namespace kvc {

const RowsKernelInfo *KVC_RCAT(KVC_TAG, KVC_INST_D)() { return rows_tc_info<KVC_ELEM, KVC_INST_D>(); }

}  // namespace kvc
