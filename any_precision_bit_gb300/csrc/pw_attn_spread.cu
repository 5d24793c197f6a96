// pw_attn_spread.cu -- the attention kernel with at most 32 query rows: single tokens.
#include "pw_attn.cuh"

namespace pw {
template int launch_form<kSpread>(const AttnArgs &, const AttnMaps &, int, cudaStream_t);
}
