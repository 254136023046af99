// Attention over shared prefixes: its forms of the cache attention's kernels (a
// file of their own, so that they compile beside the plain ones).
#include "dev_attend_pages.cuh"

namespace mk {

AttFn att_shared_kernel(AttKind kind, int D, int P, int rt) {
    return kind == ATT_OWN ? att_kernel_of<ATT_OWN>(D, P, rt) : att_kernel_of<ATT_GROUPS>(D, P, rt);
}
AttFn att_shared_merge(int D, int P, int rt) { return att_merge_of<ATT_OWN>(D, P, rt); }

}  // namespace mk
