// Block-scaled products of e4m3 (A) with e4m3 (B).
#define DG_TA 0
#define DG_TB 0
#define DG_LAUNCH launch_block_e4m3_e4m3
#include "inst_block.inc"
