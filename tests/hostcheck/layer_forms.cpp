// The rules of layer_forms.h for ctypes.
#include "../../quantized_linear_layers_token_amd/csrc/layer_forms.h"

extern "C" int heads_lanes(int dim) { return qlin::heads_lanes(dim); }
extern "C" int heads_tokens(int lanes, int heads, int64_t T) { return qlin::heads_tokens(lanes, heads, T); }
extern "C" int attn_channels(int dim) { return qlin::attn_channels(dim); }
extern "C" int attn_alone(int64_t sequences, int64_t tokens, int groups, int dim) { return qlin::attn_alone(sequences, tokens, groups, dim); }
