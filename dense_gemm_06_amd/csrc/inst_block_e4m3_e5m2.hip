// Block-scaled products of e4m3 (A) with e5m2 (B).
#define DG_TA 0
#define DG_TB 1
#define DG_LAUNCH launch_block_e4m3_e5m2
#include "inst_block.inc"
