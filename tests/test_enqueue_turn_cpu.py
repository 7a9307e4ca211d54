"""Forwards that share a workspace enqueue one at a time; others do not wait."""
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "grouped_query_attention_fwd_b200", "csrc")

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include <vector>

#include "enqueue_turn.h"

using namespace std::chrono_literals;

int main() {
  char a[2], b;
  // Calls with one workspace: never two inside.
  std::atomic<int> inside{0}, most{0}, total{0};
  std::vector<std::thread> threads;
  for (int t = 0; t < 8; ++t)
    threads.emplace_back([&, t] {
      for (int i = 0; i < 500; ++i) {
        const gqa::EnqueueTurn turn(&a[t % 2]);
        if (t % 2 != 0) continue;  // (another one's calls come and go beside)
        const int n = ++inside;
        if (n > most) most = n;
        std::this_thread::yield();
        --inside;
        ++total;
      }
    });
  for (auto& t : threads) t.join();
  if (most != 1 || total != 4 * 500) return std::printf("most %d total %d\n", +most, +total), 1;

  // One thread stays inside, as in a launch that blocks: calls with another
  // workspace go on, one with the same waits until it is done.
  std::atomic<bool> entered{false}, leave{false}, same{false}, other{false};
  std::thread blocked([&] {
    const gqa::EnqueueTurn turn(&a[0]);
    entered = true;
    while (!leave) std::this_thread::sleep_for(1ms);
  });
  while (!entered) std::this_thread::sleep_for(1ms);
  std::thread waits([&] {
    const gqa::EnqueueTurn turn(&a[0]);
    same = true;
  });
  std::thread goes([&] {
    for (int i = 0; i < 100; ++i) const gqa::EnqueueTurn turn(&b);
    other = true;
  });
  for (int i = 0; i < 5000 && !other; ++i) std::this_thread::sleep_for(1ms);
  std::this_thread::sleep_for(50ms);
  const bool ok = other && !same;
  leave = true;
  blocked.join();
  waits.join();
  goes.join();
  if (!ok || !same) return std::printf("other %d\n", +other), 2;
  return 0;
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("turn")
    (d / "turn.cpp").write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-pthread", "-I" + CSRC,
                           str(d / "turn.cpp"), "-o", str(d / "turn")])
    return str(d / "turn")


def test_turns(program):
    r = subprocess.run([program], timeout=120, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
