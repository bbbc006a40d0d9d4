"""How a launch's CTAs take its chunks (csrc/narrow/tickets.h, which the optimiser's kernel
includes), on the CPU: threads in the CTAs' place take every chunk once, whatever the word
held that they count in."""
import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NARROW = os.path.join(ROOT, "dlrm_embedding_bag_b200", "csrc", "narrow")

MODEL = r"""
#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <memory>
#include <thread>
#include <vector>
#include "tickets.h"

static long checks = 0;
#define CHECK(c) \
  do { \
    ++checks; \
    if (!(c)) { std::printf("line %d: %s (word %u, %d chunks, %d CTAs)\n", __LINE__, #c, at, chunks, ctas); std::exit(1); } \
  } while (0)

// One launch by `ctas` threads: how often each chunk was taken, how often the word was put back.
static void launch(uint32_t at, int chunks, int ctas, bool left_raised) {
  std::atomic<uint32_t> word(at);
  std::unique_ptr<std::atomic<int>[]> taken(new std::atomic<int>[chunks + 1]);
  for (int i = 0; i <= chunks; ++i) taken[i] = 0;
  std::atomic<int> ends(0), outside(0), draws(0);
  auto cta = [&](int number) {
    if (number == 0) {  // the first one's maximum
      uint32_t was = word;
      while (was < dlrm::kDrawing && !word.compare_exchange_weak(was, dlrm::kDrawing)) {
      }
    }
    uint32_t seen = word;
    if (!dlrm::raised(seen)) word.compare_exchange_strong(seen, dlrm::kDrawing);
    for (int c = number;;) {
      const uint32_t drawn = word.fetch_add(1);
      ++draws;
      if (c < chunks) {
        if (c < 0) ++outside; else ++taken[c];
      }
      const int next = dlrm::next_chunk(drawn, chunks, ctas);
      if (dlrm::last_ticket(drawn, chunks)) {
        word = 0;
        ++ends;
      }
      if (next >= chunks) break;
      c = next;
    }
  };
  std::vector<std::thread> all;
  for (int i = 0; i < ctas; ++i) all.emplace_back(cta, i);
  for (auto& t : all) t.join();
  CHECK(outside == 0);
  if (left_raised) return;
  CHECK(ends == 1 && word == 0);
  CHECK(draws == (chunks > 0 ? chunks : 1));
  for (int i = 0; i < chunks; ++i) CHECK(taken[i] == 1);
}

int main() {
  for (int chunks : {0, 1, 2, 7, 8, 9, 100, 1000}) {
    for (int ctas : {1, 2, 8, 16}) {
      if (ctas > (chunks > 1 ? chunks : 1)) continue;  // a launch has no more of them
      for (uint32_t at : {0u, 1u, 5u, 99u, 999u, 1000u, 1001u, 2000000000u, 0x7fffffffu, 0xffffffffu, 0xfffffff0u, 0xfffffc00u, 0xc0000001u})
        for (int again = 0; again < 3; ++again) launch(at, chunks, ctas, false);
      // left raised: chunks may be missed, but none is taken that is not there
      for (uint32_t at : {0x80000000u, 0x80000001u, 0x80000064u, 0xbfffffffu, 0xc0000000u}) launch(at, chunks, ctas, true);
    }
  }
  std::printf("%ld\n", checks);
}
"""


def test_every_chunk_is_taken_once_whatever_the_word_was(tmp_path):
    src = tmp_path / "model.cpp"
    src.write_text(MODEL)
    exe = tmp_path / "model"
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-Wall", "-Werror", "-I", NARROW, str(src),
                    "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout) > 10000


def test_the_kernel_takes_its_chunks_so():
    """The word is raised and the step's count read before the first ticket is drawn, and both are
    written by the one who draws the last."""
    src = open(os.path.join(NARROW, "adamw.cu")).read()
    body = src[src.index("adamw_kernel("):]
    body = body[:body.index("\n}\n")]
    raised = re.search(r"const uint32_t seen = \*static_cast<volatile uint32_t\*>\(counter\(a\)\);\s+"
                       r"if \(!raised\(seen\)\) atomicCAS\(counter\(a\), seen, kDrawing\);\s+"
                       r"__threadfence\(\)", body)
    places = [body.index("a.step[0]"), raised.start(), raised.end()] + [body.index(s) for s in (
        "atomicAdd(counter(a), 1u)", "next_chunk(drawn, a.chunks", "last_ticket(drawn, a.chunks)",
        "*counter(a) = 0")]
    assert places == sorted(places)
    assert body.count("atomicAdd(") == body.count("counter(a) = 0") == 1
    assert src.count("step + 1") == 1 and "step[1]" not in src
