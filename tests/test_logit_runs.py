"""Runs of words that the logits' kernel works on, on the host: every word of a row has
one place, and no word, whatever the context holds, a place outside its run's table."""
import ctypes
import os
import subprocess

import pytest

from precision_transformer_gemms_gb300 import build

SOURCE = r"""
#include "logit_runs.h"
using namespace lpq;
// 0, or which rule is broken first: 1 words of a run, 2 places of foreign words, 3 places of the row's words, 4 their count
extern "C" int check_row(int v, int lead, int vec, int s, int every) {
  int64_t held = 0;
  for (int run = 0; run < run_count(v, vec, s); ++run) {
    const int first = run_first(run, s, lead), words = run_words(first, s, v);
    if (words < 0 || words > s) return 1;
    const int64_t far[] = {INT64_MIN, INT64_MIN + 1, INT64_MAX, INT32_MIN, INT32_MAX, -1, -(int64_t)lead - 1, v, v + 1, v + 5000, 1 << 20, 1ll << 32,
                           (1ll << 32) + first, (1ll << 32) + v, first - 1ll, first + (int64_t)s, v + (int64_t)s - 1, (int64_t)first + INT64_MIN};
    for (int64_t w : far) {
      const int at = run_place(w, first, words);
      if (at < -1 || at >= s || (at >= 0 && (at != w - first || w >= v))) return 2;
    }
    for (int64_t w = first < 0 ? 0 : first; w < v && w < first + (int64_t)s; w += every)
      if (run_place(w, first, words) != w - first) return 3;
    const int64_t from = first < 0 ? 0 : first, to = (int64_t)first + words;
    held += to > from ? to - from : 0;
  }
  return held == v ? 0 : 4;
}
// Entries that lane `lane` of a warp reads of a list of `count` from `from` to `to`, the
// first and every one of its steps: 0, or 1 where one lies outside the list.
extern "C" int check_list(int64_t from, int64_t to, int64_t count, int lane) {
  from = within(from, count), to = within(to, count);
  for (int step = 0;; ++step) {
    const uint64_t at = (uint64_t)from + (uint64_t)lane;  // (as the device adds: modulo 2^64)
    if ((int64_t)at < to && ((int64_t)at < 0 || (int64_t)at >= count)) return 1;
    if (from >= to) return 0;
    from += 32;
  }
}
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    folder = tmp_path_factory.mktemp("runs")
    (folder / "runs.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + build.CSRC, str(folder / "runs.cpp"), "-o",
                    str(folder / "runs.so")], check=True)
    return ctypes.CDLL(os.path.join(folder, "runs.so"))


@pytest.mark.parametrize("vec,s", [(4, 1024), (4, 4096), (4, 8192), (8, 2048), (8, 4096), (8, 8192), (1, 1024), (1, 4096)])
def test_every_length_and_lead(host, vec, s):
    for v in list(range(1, 3 * s + 2 * vec)) + [50174, 50175, 131071, 131072, 131073, (1 << 30) - 1, 1 << 30]:
        near = v % s < 2 * vec or v % s > s - 2 * vec
        if v > 1 << 20 or near or v % 7 == 0:
            for lead in range(vec):
                every = 1 if near and v < 1 << 20 else 5 if v < 1 << 20 else 1001
                assert host.check_row(v, lead, vec, s, every) == 0, (v, lead)


@pytest.mark.parametrize("count", [0, 1, 31, 100])
def test_offsets_beyond_the_list(host, count):
    top = (1 << 63) - 1
    ends = [-top - 1, -top, -1000, -1, 0, 1, 31, count - 1, count, count + 1, 1 << 31, 1 << 32, top - 32, top - 31, top - 5, top]
    i64 = ctypes.c_int64
    for a in ends:
        for b in ends:
            if min(max(b, 0), count) - max(a, 0) < 1 << 20:
                for lane in (0, 5, 31):
                    assert host.check_list(i64(a), i64(b), i64(count), lane) == 0, (a, b, lane)
