// Appending to the 8-bit cache with the rotation of keys by their positions on the way, and
// the rotation of the queries.
#include "kv8_append.h"

namespace qwg {

hipError_t launch_kv8_append_rotary(Kv8RotaryArgs &a, int type, hipStream_t s) {
    // one token a sequence: a wavefront for 32 heads of it, so that all are under way at once;
    // prompts: eight heads a workgroup, under the same angles
    const bool one = a.max_new <= 1;
    a.slice = one ? 32 : 8, a.per_thread = one ? 4 : 8;
    a.rows = a.max_new < a.cache.page ? (int)a.max_new : a.cache.page;
    if (a.neighbours) {
        if (type == kF32) return append<kF32, kNeighbours>(a, s);
        if (type == kF16) return append<kF16, kNeighbours>(a, s);
        return append<kBF16, kNeighbours>(a, s);
    }
    if (type == kF32) return append<kF32, kHalves>(a, s);
    if (type == kF16) return append<kF16, kHalves>(a, s);
    return append<kBF16, kHalves>(a, s);
}

}  // namespace qwg
