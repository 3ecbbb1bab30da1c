// The adapters' kernels for bf16.
#define DG_DT dg::DT_BF16
#define DG_SUFFIX bf16
#include "inst_adapters.inc"
