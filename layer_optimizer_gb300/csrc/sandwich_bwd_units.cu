// The staged backward pass over rows on units of eight columns.
#include "sandwich_bwd_ring.cuh"

namespace sf {

const void* bwd_ring_units(int32_t ta, int32_t ts, bool kept, bool post) { return bwd_ring_of<kUnits>(ta, ts, kept, post); }

const void* device_error_sandwich_units() { return &g_device_error; }

}  // namespace sf
