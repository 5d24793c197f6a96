// pw_attn.cu -- choice of the attention kernel's form.
#include "pw_attn.h"

namespace pw {

template <int FORM, bool TREE>
int launch_form(const AttnArgs &a, const AttnMaps &maps, int bf16, cudaStream_t st);
extern template int launch_form<kTwo, false>(const AttnArgs &, const AttnMaps &, int, cudaStream_t);
extern template int launch_form<kSpread, false>(const AttnArgs &, const AttnMaps &, int, cudaStream_t);
extern template int launch_form<kTwo, true>(const AttnArgs &, const AttnMaps &, int, cudaStream_t);
extern template int launch_form<kSpread, true>(const AttnArgs &, const AttnMaps &, int, cudaStream_t);

int launch_attn(const AttnArgs &a, const AttnMaps &maps, int bf16, void *stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a.list.streams == 2)
    return a.seen ? launch_form<kTwo, true>(a, maps, bf16, st) : launch_form<kTwo, false>(a, maps, bf16, st);
  return a.seen ? launch_form<kSpread, true>(a, maps, bf16, st) : launch_form<kSpread, false>(a, maps, bf16, st);
}

}  // namespace pw
