// pw_attn_spread_tree.cu -- the attention kernel with at most 16 query rows to a tile, for small trees of drafted tokens.
#include "pw_attn.cuh"

namespace pw {
template int launch_form<kSpread, true>(const AttnArgs &, const AttnMaps &, int, cudaStream_t);
}
