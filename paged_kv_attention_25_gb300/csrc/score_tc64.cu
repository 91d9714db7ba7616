// The tensor-core form of pkv_score_attn for head_dim 64.
#include "score_tc.cuh"

template int pkv::launch_score_tc<64>(const ScoreArgs&, const void*, const void*, const void*, void*);
