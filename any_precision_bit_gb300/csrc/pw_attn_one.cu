// pw_attn_one.cu -- the attention kernel with one query tile of 33 to 128 rows: short chunks and drafts.
#include "pw_attn.cuh"

namespace pw {
template int launch_form<kOne>(const AttnArgs &, const AttnMaps &, int, cudaStream_t);
}
