// seg_scratch.cuh -- how a stream's scratch of the products grows.
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace segred {

struct Scratch {
    void* ptr = nullptr;
    size_t bytes = 0;
    uint32_t gen = 0;
};

constexpr size_t kScratchAhead = size_t(256) << 20;

// `sc` holds at least `bytes` afterwards, or nothing (false).  The old buffer
// goes before the new one comes: release(ptr) and allocate(&ptr, bytes) work in
// the order of the stream.  Twice the old size, at most kScratchAhead more than
// is needed, so that calls that need a little more each time do not allocate
// each time; and where there is no memory for that, what is needed.
template <class Allocate, class Release>
bool grow_scratch(Scratch& sc, size_t bytes, Allocate allocate, Release release) {
    if (sc.bytes >= bytes) return true;
    const size_t least = std::max<size_t>(bytes, size_t(1) << 20);
    const size_t ahead = std::max(least, std::min(2 * sc.bytes, least + kScratchAhead));
    if (sc.ptr) release(sc.ptr);
    sc = Scratch();
    for (const size_t want : {ahead, least}) {
        if (allocate(&sc.ptr, want)) {
            sc.bytes = want;
            return true;
        }
        sc.ptr = nullptr;
    }
    return false;
}

}  // namespace segred
