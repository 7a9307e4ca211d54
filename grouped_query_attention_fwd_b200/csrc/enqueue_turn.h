// One forward at a time enqueues its launches with a workspace.
//
// A forward of several launches keeps scratch in the workspace between them
// (partials, item orders, keys read back), and a forward of one launch writes
// scratch there too: a call that another thread makes with the same workspace,
// on the stream that orders the two, must not come between.  Calls with
// different workspaces never wait for one another: a thread may block inside a
// launch (a full queue) for as long as its device takes.
//
// The workspaces in use form a list of the waiting calls' own stack objects:
// nothing is allocated and nothing is left behind.
#pragma once

#include <condition_variable>
#include <mutex>

namespace gqa {

class EnqueueTurn {
 public:
  explicit EnqueueTurn(const void* workspace) : workspace_(workspace) {
    std::unique_lock<std::mutex> lock(mutex());
    freed().wait(lock, [&] { return !taken(workspace); });
    next_ = first();
    first() = this;
  }
  ~EnqueueTurn() {
    {
      const std::lock_guard<std::mutex> lock(mutex());
      EnqueueTurn** at = &first();
      while (*at != this) at = &(*at)->next_;
      *at = next_;
    }
    freed().notify_all();
  }
  EnqueueTurn(const EnqueueTurn&) = delete;
  EnqueueTurn& operator=(const EnqueueTurn&) = delete;

 private:
  static std::mutex& mutex() {
    static std::mutex m;
    return m;
  }
  static std::condition_variable& freed() {
    static std::condition_variable c;
    return c;
  }
  static EnqueueTurn*& first() {
    static EnqueueTurn* head = nullptr;
    return head;
  }
  static bool taken(const void* workspace) {
    for (const EnqueueTurn* t = first(); t != nullptr; t = t->next_)
      if (t->workspace_ == workspace) return true;
    return false;
  }

  const void* workspace_;
  EnqueueTurn* next_ = nullptr;
};

}  // namespace gqa
