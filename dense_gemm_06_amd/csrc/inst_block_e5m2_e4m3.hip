// Block-scaled products of e5m2 (A) with e4m3 (B).
#define DG_TA 1
#define DG_TB 0
#define DG_LAUNCH launch_block_e5m2_e4m3
#include "inst_block.inc"
