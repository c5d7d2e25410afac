// smem_limits.h -- which dynamic shared-memory limits have been raised.  The limit is
// an attribute of a kernel on one device, so both are the key.
#pragma once

#include <algorithm>
#include <mutex>
#include <vector>

namespace tg {

class SmemLimits {
public:
    // Whether `kernel` on `device` is known to allow at least `bytes`.
    bool known(int device, const void* kernel, unsigned bytes)
    {
        std::lock_guard<std::mutex> lock(mutex_);
        const Entry* e = find(device, kernel);
        return e && bytes <= e->bytes;
    }

    void record(int device, const void* kernel, unsigned bytes)
    {
        std::lock_guard<std::mutex> lock(mutex_);
        if (Entry* e = find(device, kernel))
            e->bytes = std::max(e->bytes, bytes);
        else
            entries_.push_back({device, kernel, bytes});
    }

private:
    struct Entry {
        int device;
        const void* kernel;
        unsigned bytes;
    };

    Entry* find(int device, const void* kernel)
    {
        for (Entry& e : entries_)
            if (e.kernel == kernel && e.device == device) return &e;
        return nullptr;
    }

    std::mutex mutex_;
    std::vector<Entry> entries_;
};

}  // namespace tg
