// Block-scaled products of e5m2 (A) with e5m2 (B).
#define DG_TA 1
#define DG_TB 1
#define DG_LAUNCH launch_block_e5m2_e5m2
#include "inst_block.inc"
