// The library's growing device buffers, apart from where their memory comes from.
#pragma once

#include <stddef.h>

#include "../../include/bdlm.h"

namespace bdlm {

struct Workspace {
  void* ptr = nullptr;
  size_t cap = 0;
  bool in_graph = false;   // a caller's graph may hold ptr
};

// Grows `w` to `need` bytes and some to spare.  `mem` is the device's memory: bool wait() for all work
// on it, bool alloc(void**, size_t), void free(void*), bool zero(void*, size_t), and bool retire(void*),
// which keeps a buffer until the workspaces are released.
//
// A buffer that no graph holds is freed first, so that growing takes no more than the new one's room.
// One that a graph may hold is retired, as a replay must still find memory there; growth then at least
// doubles, where there is room for that, so that the retired buffers add up to less than the live one.
// Where there is no room to spare the new buffer is just what the call needs.
template <typename Mem>
int grow(Workspace& w, size_t need, bool zero, Mem&& mem) {
  size_t n = need + need / 4 + 4096;
  if (w.in_graph && n < 2 * w.cap) n = 2 * w.cap;
  if (w.ptr && !mem.wait()) return BDLM_ERR_CUDA;
  if (w.ptr && !w.in_graph) {
    mem.free(w.ptr);
    w = Workspace{};
  }
  void* fresh = nullptr;
  if (!mem.alloc(&fresh, n)) {
    n = need;
    if (!mem.alloc(&fresh, n)) return BDLM_ERR_NOMEM;
  }
  if (zero && !mem.zero(fresh, n)) {
    mem.free(fresh);
    return BDLM_ERR_CUDA;
  }
  if (w.ptr && !mem.retire(w.ptr)) {
    mem.free(fresh);
    return BDLM_ERR_NOMEM;
  }
  w.ptr = fresh;
  w.cap = n;
  w.in_graph = false;
  return BDLM_OK;
}

}  // namespace bdlm
