// The staged backward pass over rows of any alignment.
#include "sandwich_bwd_ring.cuh"

namespace sf {

const void* bwd_ring_strided(int32_t ta, int32_t ts, bool kept, bool post) { return bwd_ring_of<kStrided>(ta, ts, kept, post); }

const void* device_error_sandwich_strided() { return &g_device_error; }

}  // namespace sf
