// The prompt kernel as the launchers of this library call it: for kda_attn_fwd, and for
// the shared prefix of kda_attn_step, whose rows are the queries of one sequence.
#pragma once

#include "kda_internal.h"

namespace kda {

struct AttnParts {
  float* o;        // [splits, B * T, HQ, D] fp32, normalised; nullptr: the results go to the call's o
  float* lse;      // [splits, B * T, HQ], in powers of two; -inf without a key (o: 0), and with keys that all score -inf (o: NaN)
  int splits;      // the keys' blocks are split over this many results
  int keys;        // paged keys of the one sequence, where no seq_lens_k gives them
};

// Query tokens that a CTA takes at once, and of how many query heads of a key head's group.
struct AttnTiles {
  int tokens, heads;
};
AttnTiles attn_tiles(int group);
cudaError_t launch_attn_prompts(const kda_attn_fwd_args& a, const AttnParts& parts, cudaStream_t s);

}  // namespace kda
