"""The bounded wait of the chunk kernels gives a warp one answer.  A lane may see a barrier
complete at another try than its neighbour (the instruction does not promise that lanes
agree), while another warp calls the kernel off: lanes that parted there would meet
full-warp shuffles, products and block barriers alone.  The wait's own source is compiled
for the host with 32 threads as lanes and votes that join them."""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "offloaded_kv_cache_gb300", "csrc")

HOST = r"""
#include <atomic>
#include <barrier>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <thread>
#include <vector>
#define __device__
#define __forceinline__ inline
constexpr int kLanes = 32;
thread_local int lane, tries;
int scenario;
std::barrier<> meet(kLanes);
std::atomic<int> votes{0};
volatile int called_off;
bool vote(bool p, bool all) {
  meet.arrive_and_wait();
  if (lane == 0) votes = 0;
  meet.arrive_and_wait();
  votes += p;
  meet.arrive_and_wait();
  const bool r = all ? votes == kLanes : votes > 0;
  meet.arrive_and_wait();
  return r;
}
bool __all_sync(unsigned, int p) { return vote(p, true); }
bool __any_sync(unsigned, int p) { return vote(p, false); }
bool mbar_try_wait(uint32_t, uint32_t) {
  const int n = tries++;
  switch (scenario) {
    case 0: return true;                        // complete
    case 1: return lane % 2 == 0;               // some lanes see it, others do not yet
    case 2: return lane % 2 == 0 || n >= 3;     // they do at a later try
    case 3: return lane != 5 || n >= 2;         // one lane is late
    default: return false;                      // it never completes
  }
}
// case 5: one lane's clock runs out before the others'
uint64_t global_ns() { return (scenario != 5 || lane == 7) ? 1000ull * tries : 0; }
@WAITER@
int main(int argc, char **argv) {
  scenario = atoi(argv[1]);
  called_off = atoi(argv[2]);  // by another warp
  std::vector<int> got(kLanes, -1);
  std::vector<std::thread> t;
  for (int i = 0; i < kLanes; ++i)
    t.emplace_back([&got, i] {
      lane = i;
      tries = 0;
      const Waiter wait{&called_off, 5000};
      got[i] = wait(0, 0);
    });
  for (auto &x : t) x.join();
  for (int g : got) printf("%d ", g);
  printf("%d\n", (int)called_off);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    with open(os.path.join(CSRC, "kv_chunk.cuh")) as f:
        struct = re.search(r"^struct Waiter \{.*?^\};", f.read(), re.S | re.M).group(0)
    struct = re.sub(r"#pragma unroll.*", "", struct)
    d = tmp_path_factory.mktemp("wait")
    (d / "wait.cpp").write_text(HOST.replace("@WAITER@", struct))
    subprocess.run(["g++", "-std=c++20", "-O1", "-pthread", "-o", str(d / "wait"),
                    str(d / "wait.cpp")], check=True)
    return str(d / "wait")


@pytest.mark.parametrize("scenario,called_off,answer", [
    (0, 0, 1), (0, 1, 1), (1, 1, 0), (1, 0, 0), (2, 0, 1), (2, 1, 0), (3, 0, 1), (3, 1, 0),
    (4, 0, 0), (4, 1, 0), (5, 0, 0)])
def test_a_warp_has_one_answer(program, scenario, called_off, answer):
    r = subprocess.run([program, str(scenario), str(called_off)], capture_output=True, text=True,
                       timeout=60, check=True)
    *got, off = [int(x) for x in r.stdout.split()]
    assert got == [answer] * 32
    assert off == (called_off or not answer)  # who gives up calls the kernel off
