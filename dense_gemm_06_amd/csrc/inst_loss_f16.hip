// The loss's kernels for fp16.
#define DG_DT dg::DT_F16
#define DG_SUFFIX f16
#include "inst_loss.inc"

namespace dg {

int launch_loss_turn(const void* x, int64_t ldx, int tokens, int cols, void* out, int64_t ld, hipStream_t s) {
    const TurnArgs t{x, ldx, 0, tokens, cols, out, (int)ld, pieces<64>((int)ld), pieces<64>(cols)};
    return launch_status(loss_turn, dim3((unsigned)(t.tiles_r * t.tiles_c)), dim3(256), s, t);
}

int launch_loss_finish(const void* part, int strips, int tokens, const int64_t* target, int vocabulary,
                       const float* picked, float* loss, float* lse, hipStream_t s) {
    // up to 256 workgroups before a workgroup gets more than one token (64 tokens, 2048 strips: 32.8 to
    // 18.6 us for the whole call against 64 tokens to a workgroup, 16 tokens: 29.5 to 27.5)
    int width = 1;
    while (width < 64 && (int64_t)width * 256 < tokens) width *= 2;
    return launch_status(loss_finish, dim3((unsigned)((tokens + width - 1) / width)), dim3(1024), s,
                         static_cast<const LossPart*>(part), strips, tokens, width, target, vocabulary, picked, loss, lse);
}

}  // namespace dg
