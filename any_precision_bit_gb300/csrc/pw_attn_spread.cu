// pw_attn_spread.cu -- the attention kernel with at most 16 query rows to a tile: single tokens and drafts.
#include "pw_attn.cuh"

namespace pw {
template int launch_form<kSpread>(const AttnArgs &, const AttnMaps &, int, cudaStream_t);
}
