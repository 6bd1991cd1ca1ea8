// fa_workspace.h -- the device memory that the library keeps for the streams it is
// called on (internal; host only, no CUDA header: Api makes the calls).
#pragma once
#include <cstddef>
#include <mutex>
#include <vector>

namespace fa {

// One block of memory per stream: calls on one stream run in order, calls on
// different streams may overlap.  A stream is known by its id, which is unique for
// the life of the program.  Its handle is not: cudaStreamPerThread names another
// stream in every thread, and a destroyed stream's handle may return as a new
// stream's, while the old one's last work still runs.
//
// Api: Stream, the handle's type; id(stream, &id) and alloc(&ptr, bytes), false on
// failure; free(ptr), which waits for the work that uses the memory, false on
// failure; shared(stream): other threads' streams have this handle too.
template <class Api>
class StreamWorkspaces {
 public:
  using Stream = typename Api::Stream;
  struct Entry {
    unsigned long long id;
    Stream stream;
    void* ptr = nullptr;
    size_t bytes = 0;
    // the pair kernel's tail-split arrival counters: a block of their own (no other
    // call writes it), zeroed when made, and the epoch of the last launch that
    // used them on this stream
    void* tail_ctr = nullptr;
    size_t tail_ctr_n = 0;
    unsigned tail_epoch = 0;
  };

  // The stream's entry with at least `need` bytes; null on failure.  It stays in
  // place until the next call.
  Entry* get(Stream stream, size_t need) {
    unsigned long long id = 0;
    if (!Api::id(stream, &id)) return nullptr;
    for (Entry& e : all_)
      if (e.id == id) return grow(e, need) ? &e : nullptr;
    if (!Api::shared(stream)) {
      for (size_t i = 0; i < all_.size(); ++i) {
        if (all_[i].stream != stream) continue;  // else the handle of a destroyed stream
        drop(all_[i]);
        all_.erase(all_.begin() + static_cast<std::ptrdiff_t>(i));
        break;
      }
    }
    Entry e{};
    e.id = id;
    e.stream = stream;
    if (!grow(e, need)) return nullptr;
    all_.push_back(e);
    return &all_.back();
  }

  // Frees every entry's memory; false if a free failed.
  bool release() {
    bool ok = true;
    for (Entry& e : all_) ok = drop(e) && ok;
    all_.clear();
    return ok;
  }

  // The memory went away with its context.
  void forget() { all_.clear(); }

 private:
  static bool grow(Entry& e, size_t need) {
    if (e.bytes >= need) return true;
    if (e.ptr) Api::free(e.ptr);
    e.ptr = nullptr;
    e.bytes = 0;
    if (!Api::alloc(&e.ptr, need)) {
      e.ptr = nullptr;
      return false;
    }
    e.bytes = need;
    return true;
  }
  static bool drop(Entry& e) {
    bool ok = true;
    if (e.ptr) ok = Api::free(e.ptr) && ok;
    if (e.tail_ctr) ok = Api::free(e.tail_ctr) && ok;
    return ok;
  }

  std::vector<Entry> all_;
};

// Every device's, each behind a lock of its own: an allocation or a free, which
// waits for its device, keeps no call on another device waiting.
template <class Api, int kDevices>
class DeviceWorkspaces {
 public:
  using Streams = StreamWorkspaces<Api>;

  // The entry of a stream of device `dev` (see StreamWorkspaces::get).  `hold` is
  // locked on return, and no other call gets at the device's entries until it is
  // given up.
  typename Streams::Entry* acquire(int dev, typename Api::Stream stream, size_t need,
                                   std::unique_lock<std::mutex>* hold) {
    *hold = std::unique_lock<std::mutex>(at_[dev].mu);
    return at_[dev].streams.get(stream, need);
  }
  std::unique_lock<std::mutex> lock(int dev) { return std::unique_lock<std::mutex>(at_[dev].mu); }
  // With the device's lock held: frees its memory; false if a free failed.
  bool release(int dev) { return at_[dev].streams.release(); }
  void forget(int dev) {
    std::lock_guard<std::mutex> lock(at_[dev].mu);
    at_[dev].streams.forget();
  }

 private:
  struct Device {
    std::mutex mu;
    Streams streams;
  };
  Device at_[kDevices];
};

}  // namespace fa
