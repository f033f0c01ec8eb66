// The library-owned workspaces, one per (device, stream).  Plain C++17 with no
// HIP types, so that the same code is compiled into the library
// (nvfp4_gemv.hip) and into a host-only check built with g++ and the address and
// undefined-behaviour sanitizers.  Not part of the C ABI.
#ifndef NVFP4_WORKSPACE_TABLE_H
#define NVFP4_WORKSPACE_TABLE_H

#include <cstddef>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

namespace nvfp4ws {

// A slot only grows.  Growing allocates a new buffer and retires the old one
// without freeing it: kernels enqueued earlier on the stream may still read it,
// and freeing it safely would need a synchronisation.  Retired buffers are kept
// until the process ends; each growth at least doubles the slot, so they add
// at most the slot's final size.  No allocation is made while the stream is
// being captured into a graph (the call fails instead).
class WorkspaceTable {
public:
    // At least `need` bytes, or nullptr when the slot must grow and cannot.
    // alloc(bytes) -> pointer or nullptr, capturing() -> whether the stream is being
    // captured; neither may throw.  The table's own exceptions (host memory runs out)
    // end here, since the callers are C entry points.
    template <typename Alloc, typename Capturing>
    void *get(int dev, void *stream, size_t need, Alloc alloc, Capturing capturing) noexcept {
        try {
            std::lock_guard<std::mutex> lock(mutex_);
            auto &slot = slots_[std::make_pair(dev, stream)];
            if (slot.second >= need) return slot.first;
            if (capturing()) return nullptr;
            retired_.reserve(retired_.size() + 1);   // before there is a buffer to lose
            size_t bytes = slot.second > need / 2 ? 2 * slot.second : need;
            bytes = (bytes + 255) & ~size_t(255);
            void *ptr = alloc(bytes);
            if (!ptr) return nullptr;
            if (slot.first) retired_.push_back(slot.first);
            slot = std::make_pair(ptr, bytes);
            return ptr;
        } catch (...) {
            return nullptr;
        }
    }

private:
    std::mutex mutex_;
    std::map<std::pair<int, void *>, std::pair<void *, size_t>> slots_;
    std::vector<void *> retired_;
};

}  // namespace nvfp4ws

#endif  // NVFP4_WORKSPACE_TABLE_H
