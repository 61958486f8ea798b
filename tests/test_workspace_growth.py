"""How the library's workspaces grow (csrc/workspace.h), against a device memory of the test's own:
what is freed, kept and asked for, and which failures leave what behind."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHECK = r"""
#include <stdio.h>
#include <stdlib.h>
#include <map>
#include <vector>
#include "workspace.h"

#define CHECK(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); exit(1); } } while (0)

struct Fake {   // room for `room` bytes; addresses are never used twice
  size_t room;
  std::map<size_t, size_t> live;
  std::vector<size_t> kept, asked;
  size_t next = 4096;
  int waits = 0, fail_zero = 0, fail_retire = 0, fail_wait = 0;
  size_t used() const { size_t s = 0; for (auto& x : live) s += x.second; return s; }
  bool wait() { ++waits; return !fail_wait; }
  bool alloc(void** p, size_t n) {
    asked.push_back(n);
    if (used() + n > room) return false;
    live[next] = n;
    *p = reinterpret_cast<void*>(next);
    next += 4096;
    return true;
  }
  void free(void* p) { CHECK(live.erase(reinterpret_cast<size_t>(p)) == 1); }
  bool zero(void* p, size_t n) { CHECK(live.at(reinterpret_cast<size_t>(p)) == n); return !fail_zero; }
  bool retire(void* p) { if (fail_retire) return false; kept.push_back(reinterpret_cast<size_t>(p)); return true; }
};

int main() {
  using bdlm::Workspace;
  using bdlm::grow;
  const size_t M = 1 << 20;
  {   // the first allocation has room to spare and waits for nothing
    Fake f{100 * M};
    Workspace w;
    CHECK(grow(w, 10 * M, true, f) == BDLM_OK && w.cap == 10 * M + 10 * M / 4 + 4096 && f.waits == 0);
    // growth that no graph has seen: the old buffer is gone, nothing doubles
    CHECK(grow(w, 13 * M, false, f) == BDLM_OK && w.cap == 13 * M + 13 * M / 4 + 4096);
    CHECK(f.live.size() == 1 && f.kept.empty() && f.waits == 1 && !w.in_graph);
    // it fits although both buffers together do not
    CHECK(grow(w, 75 * M, false, f) == BDLM_OK && f.live.size() == 1);
    // no room to spare: just what is needed
    CHECK(grow(w, 99 * M, false, f) == BDLM_OK && w.cap == 99 * M && f.live.size() == 1);
    // no room: the workspace is empty, and serves what fits again
    CHECK(grow(w, 101 * M, false, f) == BDLM_ERR_NOMEM && w.ptr == nullptr && w.cap == 0 && f.live.empty());
    CHECK(grow(w, 20 * M, false, f) == BDLM_OK && f.live.size() == 1);
  }
  {   // a buffer that a graph holds stays, and growth doubles
    Fake f{100 * M};
    Workspace w;
    CHECK(grow(w, 10 * M, false, f) == BDLM_OK);
    void* first = w.ptr;
    const size_t cap = w.cap;
    w.in_graph = true;
    CHECK(grow(w, 13 * M, false, f) == BDLM_OK && w.cap == 2 * cap && w.ptr != first && !w.in_graph);
    CHECK(f.kept.size() == 1 && f.kept[0] == reinterpret_cast<size_t>(first) && f.live.size() == 2);
    // the larger one, which no graph has seen, is given back when it grows in its turn
    CHECK(grow(w, 30 * M, false, f) == BDLM_OK && f.live.size() == 2 && f.kept.size() == 1);
    // no room for twice as much, but for what is needed
    w.in_graph = true;
    CHECK(grow(w, 45 * M, false, f) == BDLM_OK && w.cap == 45 * M && f.kept.size() == 2);
    // no room: a graph's buffer stays and goes on serving
    w.in_graph = true;
    void* now = w.ptr;
    CHECK(grow(w, 60 * M, false, f) == BDLM_ERR_NOMEM && w.ptr == now && w.cap == 45 * M && w.in_graph);
  }
  {   // other failures leak nothing
    Fake f{100 * M};
    Workspace w;
    f.fail_zero = 1;
    CHECK(grow(w, M, true, f) == BDLM_ERR_CUDA && f.live.empty() && w.ptr == nullptr && w.cap == 0);
    f.fail_zero = 0;
    CHECK(grow(w, M, true, f) == BDLM_OK);
    w.in_graph = true;
    f.fail_retire = 1;
    void* now = w.ptr;
    CHECK(grow(w, 9 * M, true, f) == BDLM_ERR_NOMEM && f.live.size() == 1 && w.ptr == now && w.in_graph);
    f.fail_wait = 1;
    CHECK(grow(w, 9 * M, true, f) == BDLM_ERR_CUDA && f.live.size() == 1 && w.ptr == now);
  }
  printf("fine\n");
}
"""


def test_growth(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    (tmp_path / "check.cpp").write_text(CHECK)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "block_diffusion_gb300", "csrc"),
                    str(tmp_path / "check.cpp"), "-o", str(tmp_path / "check")], check=True, timeout=120)
    r = subprocess.run([str(tmp_path / "check")], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stdout
