// The loss's kernels for bf16.
#define DG_DT dg::DT_BF16
#define DG_SUFFIX bf16
#include "inst_loss.inc"
