// pw_attn_two_tree.cu -- the attention kernel with two query tiles to a CTA, for trees of drafted tokens.
#define PW_RARE __forceinline__
#include "pw_attn.cuh"

namespace pw {
template int launch_form<kTwo, true>(const AttnArgs &, const AttnMaps &, int, cudaStream_t);
}
