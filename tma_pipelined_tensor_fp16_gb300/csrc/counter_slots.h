// counter_slots.h -- which of a device's tile counters a run uses.  Runs that may be on
// the GPU at the same time must not share one: runs on one stream never are, whatever
// their plans, runs on two streams may be, and a launch captured into a graph may be
// replayed beside any other.  So every stream has a counter, and every captured launch
// one of its own for as long as its graph lives.
#pragma once

#include <cstdint>
#include <mutex>
#include <vector>

namespace tg {

class CounterSlots {
public:
    static constexpr int STREAMS = 256;    // counters of streams: the first ones
    static constexpr int CAPTURES = 65280; // counters of captured launches
    static constexpr int COUNT = STREAMS + CAPTURES;

    CounterSlots()
    {
        streams_.reserve(STREAMS);
        free_.reserve(CAPTURES);  // release() never allocates
    }

    // The counter of the stream with this id (ids are never used again).  With more
    // streams than counters the one unused for longest is taken over, and `*taken_over`
    // says so: the caller lets the device finish before it uses it.
    int of_stream(uint64_t id, bool* taken_over)
    {
        std::lock_guard<std::mutex> lock(mutex_);
        *taken_over = false;
        size_t oldest = 0;
        for (size_t i = 0; i < streams_.size(); ++i) {
            if (streams_[i].id == id) {
                streams_[i].used = ++clock_;
                return static_cast<int>(i);
            }
            if (streams_[i].used < streams_[oldest].used) oldest = i;
        }
        if (streams_.size() < STREAMS) {
            streams_.push_back({id, ++clock_});
            return static_cast<int>(streams_.size()) - 1;
        }
        *taken_over = true;
        streams_[oldest] = {id, ++clock_};
        return static_cast<int>(oldest);
    }

    // The device could not be waited for: the counter is nobody's, and the next one to
    // be taken over.
    void give_up(int slot)
    {
        std::lock_guard<std::mutex> lock(mutex_);
        streams_[static_cast<size_t>(slot)] = {NOBODY, 0};
    }

    // A counter for a launch that is being captured; -1: none left.
    int of_capture()
    {
        std::lock_guard<std::mutex> lock(mutex_);
        if (!free_.empty()) {
            const int slot = free_.back();
            free_.pop_back();
            return slot;
        }
        return captured_ < CAPTURES ? STREAMS + captured_++ : -1;
    }

    // The graph that held the counter is gone.
    void release(int slot)
    {
        std::lock_guard<std::mutex> lock(mutex_);
        free_.push_back(slot);
    }

private:
    static constexpr uint64_t NOBODY = ~uint64_t(0);
    struct Stream {
        uint64_t id, used;
    };
    std::mutex mutex_;
    std::vector<Stream> streams_;
    std::vector<int> free_;
    uint64_t clock_ = 0;
    int captured_ = 0;
};

}  // namespace tg
