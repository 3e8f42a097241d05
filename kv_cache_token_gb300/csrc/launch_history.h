// What the host has launched, for programmatic dependent launch: which decode
// kernels may start before the kernel in front of them has finished.
//
// An attention kernel checks on the device, before it writes anything, that
// every decode epilogue launched earlier on its scratch copy has finished
// (which also covers every earlier epilogue of its own layer, which uses the
// same copy), so it may start early after any kernel but two: a separate apply
// kernel, which rewrites a layer's tables after its epilogue has finished and
// lets its successor start at once, and one that writes a step's queries, keys
// and values, which the attention reads at once.  Early start concerns the
// kernel in front in the same stream only, so those two hold their stream until
// another kernel has been launched there (it waits for them); launches on other
// streams change nothing.  The epilogue starts early only right after its
// layer's attention launch.
//
// Host code without CUDA types (a stream is an address), so that its rules can
// be tested without a GPU.  Calls may come from several host threads.
#pragma once
#include <mutex>

namespace kve {

class LaunchHistory {
 public:
  // an attention, an epilogue, an apply kernel, one that writes a step's inputs, any other
  void attend(int layer, const void* stream) { note(kAttend, layer, stream, false); }
  void epilogue(int layer, const void* stream) { note(kEpilogue, layer, stream, false); }
  void apply(const void* stream) { note(kOther, -1, stream, true); }
  void inputs(const void* stream) { note(kOther, -1, stream, true); }
  // launched: the kernel is in the stream (a failed launch has put nothing behind what is there)
  void other(const void* stream, bool launched) {
    if (launched) {
      note(kOther, -1, stream, false);
    } else {
      const std::lock_guard<std::mutex> lock(mu_);
      last_ = kOther;
    }
  }

  bool attend_early(const void* stream) const {
    const std::lock_guard<std::mutex> lock(mu_);
    return !all_held_ && find(key(stream)) == n_held_;
  }
  bool epilogue_early(int layer) const {
    const std::lock_guard<std::mutex> lock(mu_);
    return last_ == kAttend && last_layer_ == layer;
  }

 private:
  enum Kind { kOther, kAttend, kEpilogue };
  static constexpr int kMost = 128;     // held streams at a time; with more, nothing starts early any more

  // the legacy default stream has two handles, 0 and 1
  static const void* key(const void* stream) {
    return stream == reinterpret_cast<const void*>(1) ? nullptr : stream;
  }
  int find(const void* k) const {
    int i = 0;
    while (i < n_held_ && held_[i] != k) ++i;
    return i;
  }
  void note(Kind kind, int layer, const void* stream, bool hold) {
    const std::lock_guard<std::mutex> lock(mu_);
    last_ = kind;
    last_layer_ = layer;
    const int i = find(key(stream));
    if (hold && i == n_held_) {
      if (n_held_ == kMost) all_held_ = true;
      else held_[n_held_++] = key(stream);
    } else if (!hold && i < n_held_) {
      held_[i] = held_[--n_held_];
    }
  }

  mutable std::mutex mu_;
  Kind last_ = kOther;
  int last_layer_ = -1;
  const void* held_[kMost] = {};
  int n_held_ = 0;
  bool all_held_ = false;
};

}  // namespace kve
