// The adapters' kernels for fp16, and their choice by type.
#define DG_DT dg::DT_F16
#define DG_SUFFIX f16
#include "inst_adapters.inc"

namespace dg {

int launch_adapter_turn(const TurnArgs& p, const TurnArgs& q, int adapters, hipStream_t s) {
    const dim3 grid((unsigned)(p.tiles_r * p.tiles_c + q.tiles_r * q.tiles_c), (unsigned)adapters);
    return launch_status(adapter_turn, grid, dim3(256), s, p, q);
}

}  // namespace dg
