// kv8_seen.cuh -- which tiles of positions a CTA's query rows see, through a window with sinks.
#pragma once

namespace bsg {
namespace {

// What a CTA of some rows sees: the tiles from `first`, then (whose few positions would
// begin with a low reference) `sink_tiles` from the sequence's start.
struct Seen {
    int tiles, sink_tiles, first;
    int low, see;  // the lowest position of the window part, and the end
    __device__ __forceinline__ int tile(int i) const {
        const int near = tiles - sink_tiles;
        return i < near ? first + i : i - near;
    }
};
template <int kN>
__device__ __forceinline__ Seen seen_by(int first_pos, int last_pos, int window, int sinks) {
    Seen s;
    s.see = last_pos + 1;
    s.low = window && first_pos >= window ? first_pos - window + 1 : 0;
    if (s.see <= 0) {
        s.tiles = s.sink_tiles = s.first = 0;
        return s;
    }
    const int k = min(sinks, s.low);
    s.sink_tiles = (k + kN - 1) / kN;
    s.first = max(s.sink_tiles, s.low / kN);
    s.tiles = s.sink_tiles + max(0, (s.see + kN - 1) / kN - s.first);
    return s;
}

}  // namespace
}  // namespace bsg
