// pw_attn_two.cu -- the attention kernel with two query tiles to a CTA.
#define PW_RARE __forceinline__
#include "pw_attn.cuh"

namespace pw {
template int launch_form<kTwo, false>(const AttnArgs &, const AttnMaps &, int, cudaStream_t);
}
