// The gated feed-forward block H = act(X Wg^T) (.) (X Wu^T) for one token,
// two tokens, and up to eight tokens on large layers (gfx950): the fp4 x fp8
// matrix-core products of f4_forms.h on the stacked layer, whose 16-row tiles
// hold 8 gate rows and the same 8 up rows, with the activation and the
// product applied where a tile's wavefront sums are added.  The two
// projections, the activation and the product are one kernel and the fp32
// pre-activations never leave it.  Bound as there by the read of the signs (two
// 11008 x 4096, K = 3: 8.6 us for one token, 38 MB; 13.9 us for 8 tokens,
// where the bf16 +-1 kernel takes 20.6).
#include "f4_forms.h"
#include "mbok_gated.h"

namespace mbok {

int gated_f4_max_tokens() { return kF4gTokens; }

int launch_gated_f4(const mbok_desc* stacked, const void* packed, const void* X, int64_t T,
                    int64_t ldx, const GatedOut& out, hipStream_t stream) {
  return launch_f4_forms(stacked, packed, X, T, ldx, out, stream);
}

}  // namespace mbok
