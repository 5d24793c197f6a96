// pw_attn.cu -- choice of the attention kernel's form.
#include "pw_attn.h"

namespace pw {

template <int FORM>
int launch_form(const AttnArgs &a, const AttnMaps &maps, int bf16, cudaStream_t st);
extern template int launch_form<kTwo>(const AttnArgs &, const AttnMaps &, int, cudaStream_t);
extern template int launch_form<kSpread>(const AttnArgs &, const AttnMaps &, int, cudaStream_t);

int launch_attn(const AttnArgs &a, const AttnMaps &maps, int bf16, void *stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return a.list.streams == 2 ? launch_form<kTwo>(a, maps, bf16, st) : launch_form<kSpread>(a, maps, bf16, st);
}

}  // namespace pw
