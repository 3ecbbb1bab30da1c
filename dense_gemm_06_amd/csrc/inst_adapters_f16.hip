// The adapters' kernels for fp16.
#define DG_DT dg::DT_F16
#define DG_SUFFIX f16
#include "inst_adapters.inc"
