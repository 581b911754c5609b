// The layer Y = R + act(X W_hat^T + b) for one token, two tokens, and up to
// eight tokens on large layers (gfx950): the fp4 x fp8 matrix-core products of
// f4_forms.h with bias, activation and residual applied where a tile's
// wavefront sums are added.  Bound as there by the read of the signs.  (4096 x
// 11008, K = 3, one token with the residual: 6.3 us in a graph, 17.9 MB; 16 tokens of 11008 x
// 4096 on the few-token kernel with bias and gelu 13.2.)
#include "f4_forms.h"
#include "mbok_linear.h"

namespace mbok {

int launch_linear_f4(const mbok_desc* d, const void* packed, const void* X, int64_t T,
                     int64_t ldx, const LinearOut& out, hipStream_t stream) {
  return launch_f4_forms(d, packed, X, T, ldx, out, stream);
}

}  // namespace mbok
