// Tensor maps (TMA descriptors) for the operand tiles of the projection (2-D, rows
// of any matrix) and for the per-chunk input tiles of the fused chunk kernel: one
// 3-D map [tokens][heads][channels] per input, box 16 tokens x 1 head x 128
// channels, rows past the end read as zero.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "kda_internal.h"

namespace kda {

struct TmaInputMaps {
  CUtensorMap q, k, v, a;  // a: gate inputs or log-decay g (fp32); unused without a gate
};

// Host: fills the maps for a bf16 dk = dv = 128 call. Returns cudaErrorInvalidValue
// if the driver cannot encode them.
cudaError_t encode_input_maps(const ChunkCall& c, TmaInputMaps* m);

// Host: a 2-D map of a [rows, cols] matrix with row stride ld (elements of 1 or 2
// bytes; base and pitch 16-byte aligned), box box_rows x 128 bytes in the 128-byte
// swizzle; rows and columns past the ends read as zero.
bool encode_rows(CUtensorMap* m, const void* base, size_t elem, long long cols, long long rows, long long ld,
                 unsigned box_rows);

// Host: a 3-D map [rows][heads][D] of bf16 (strides in elements; base and strides 16-byte
// aligned), box box_rows x box_heads x 64 channels in the 128-byte swizzle; places past
// the ends read as zero.
bool encode_heads(CUtensorMap* m, const void* base, int D, long long heads, long long head_stride, long long rows, long long row_stride,
                  unsigned box_heads, unsigned box_rows);

}  // namespace kda
