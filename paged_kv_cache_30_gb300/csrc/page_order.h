// page_order.h -- which kernels need a memset before them because a page call came before.
//
// The page calls write block tables, lengths and pages, and some attention kernels read those
// before their dependency wait (programmatic dependent launch).  Programmatic dependence
// holds between neighbouring kernels of a stream alone, so a memset between the two makes
// the second start after the first has ended.  This class keeps, on the host, the streams
// where one is due.  Its caller puts each call into the stream under the same lock as the
// entry (or the question) here.
//
// What is enqueued and what a capture records are apart: a graph runs when it is launched,
// behind all work of its stream, so a capture neither settles an enqueued page call nor leaves
// one behind.  Within a capture a kernel can also follow a page call of another stream (joined
// by an event), and the capture may make that edge programmatic as well: with page calls on
// another stream of the same capture every kernel gets its memset.
#pragma once

namespace pkv {

class PageOrder {
 public:
  static constexpr int kStreams = 64;  // kept at most

  // A page call's last kernel is in `stream` (capture: 0, or the id of the stream's capture).
  // True: there is no room to remember it, and the caller puts the memset in now.
  bool wrote(const void* stream, unsigned long long capture) {
    if (per_thread(stream)) return true;  // one handle, a stream for each thread
    stream = base(stream);
    for (int i = 0; i < n_; ++i)
      if (entries_[i].stream == stream && (entries_[i].capture != 0) == (capture != 0)) {
        // a stream is in one capture at a time: an entry of an earlier one is of no more use
        entries_[i].capture = capture;
        entries_[i].due = true;
        return false;
      }
    if (n_ == kStreams) return true;
    entries_[n_++] = {stream, capture, true};
    return false;
  }

  // Whether a kernel that reads ahead of its wait needs the memset when it goes into `stream`.
  bool due(const void* stream, unsigned long long capture) const {
    if (per_thread(stream)) return false;
    stream = base(stream);
    bool need = false;
    for (int i = 0; i < n_; ++i) {
      const Entry& e = entries_[i];
      if (e.capture == capture) need |= e.stream == stream ? e.due : capture != 0;
    }
    return need;
  }

  // The memset is in `stream`, or a kernel that waits before it reads and before it lets the
  // next one start: nothing is due on the stream any more.
  void settled(const void* stream, unsigned long long capture) {
    stream = base(stream);
    for (int i = 0; i < n_; ++i)
      if (entries_[i].stream == stream && entries_[i].capture == capture) {
        entries_[i].due = false;
        if (capture == 0) entries_[i] = entries_[--n_];
        return;
      }
  }

  bool settle(const void* stream, unsigned long long capture) {
    const bool need = due(stream, capture);
    settled(stream, capture);
    return need;
  }

  int size() const { return n_; }

 private:
  struct Entry {
    const void* stream;
    unsigned long long capture;
    bool due;
  };
  // cudaStreamLegacy is the default stream, cudaStreamPerThread another one in each thread
  static const void* base(const void* stream) {
    return stream == reinterpret_cast<const void*>(0x1) ? nullptr : stream;
  }
  static bool per_thread(const void* stream) {
    return stream == reinterpret_cast<const void*>(0x2);
  }

  Entry entries_[kStreams];
  int n_ = 0;
};

}  // namespace pkv
