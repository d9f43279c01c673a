// Host helpers that need no HIP, so that a test can compile them alone.
#pragma once

namespace qw3_host {

// Room in a vector for one more entry; false where there is no memory.  Asked for
// before push_back: no C++ exception leaves a C entry point.
template <class Vector>
bool room_for_one(Vector &v) noexcept {
    try {
        if (v.size() == v.capacity()) v.reserve(2 * v.size() + 4);
        return true;
    } catch (...) {
        return false;
    }
}

}  // namespace qw3_host
