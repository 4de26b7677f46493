// The beam search's step, for the C-ABI layer (see idx_beam_step in lidx.h).
#pragma once

#include "lidx_internal.cuh"

namespace lidx {

constexpr int kBeamMax = 1024;      // beams of a sequence
constexpr int kBeamOutMax = 32;     // continuations kept: a sort of a warp's lanes finds the bound

int64_t beam_workspace_bytes(int64_t seqs, int64_t beams, int64_t out, int64_t vocab);
cudaError_t launch_beam(const idx_beam& b, int dtype, int seqs, int beams, int out, int vocab, int end, void* ws, cudaStream_t st);

}  // namespace lidx
