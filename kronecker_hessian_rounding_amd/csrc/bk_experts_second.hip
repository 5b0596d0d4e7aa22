// bk_experts_second.hip -- the experts' second product (kernels in bk_experts.hpp).
#include "bk_experts.hpp"

namespace bk {

void launch_experts_second_few(const FewArgs& e, int W, int fs, int splits, int tiles, void* y, int ytype, int64_t ldy, hipStream_t stream) {
    if (W == 4) {
        if (fs == 1) launch_second_few<4, 1>(e, splits, tiles, y, ytype, ldy, stream);
        else launch_second_few<4, 4>(e, splits, tiles, y, ytype, ldy, stream);
    } else {
        if (fs == 1) launch_second_few<2, 1>(e, splits, tiles, y, ytype, ldy, stream);
        else launch_second_few<2, 4>(e, splits, tiles, y, ytype, ldy, stream);
    }
}

void launch_experts_second(const ExpertArgs& e, int tile, int W, int fs, hipStream_t stream) {
    if (W == 4) {
        if (fs == 1) launch_second_shape<4, 1>(e, tile, stream);
        else launch_second_shape<4, 4>(e, tile, stream);
    } else {
        if (fs == 1) launch_second_shape<2, 1>(e, tile, stream);
        else launch_second_shape<2, 4>(e, tile, stream);
    }
}

}  // namespace bk
