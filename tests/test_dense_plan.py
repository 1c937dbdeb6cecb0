"""The dense readout's work split (csrc/dense_plan.cuh) on the CPU, a warp as 32
threads: every unit of every pair is in one worker's range, and the walk ends
inside its arrays even when the lengths change under it."""
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_fp4_csa2_gb300", "csrc")

SHIM = r"""
#pragma once
#include <atomic>
#include <barrier>
#include <cstdint>
#include <vector>
#define __device__
#define __forceinline__ inline
#define __align__(n) alignas(n)
#define CSA2_DEV_ERR_NVIS 1u
struct __half;
struct __nv_bfloat16;
inline thread_local int t_lane = 0;
inline std::barrier<> g_bar(32);
inline int64_t g_x[32];
inline std::atomic<long> g_reads{0};
inline long g_change_at = -1;            // after so many reads every length is g_after
inline int g_after = 0;
inline const int32_t *g_lo = nullptr, *g_hi = nullptr;
inline std::atomic<int> g_bad{0};
inline int __ldg(const int32_t *p) {
  if (p < g_lo || p >= g_hi) { g_bad = 1; return 0; }
  const long n = g_reads++;
  return g_change_at >= 0 && n >= g_change_at ? g_after : *p;
}
inline int64_t lane_read(int64_t x, int from) {
  g_x[t_lane] = x;
  g_bar.arrive_and_wait();
  const int64_t y = from >= 0 && from < 32 ? g_x[from] : x;
  g_bar.arrive_and_wait();
  return y;
}
template <class T> T __shfl_xor_sync(unsigned, T x, int o) { return (T)lane_read(x, t_lane ^ o); }
template <class T> T __shfl_up_sync(unsigned, T x, int o) { return (T)lane_read(x, t_lane - o); }
template <class T> T __shfl_sync(unsigned, T x, int from) { return (T)lane_read(x, from); }
inline unsigned __ballot_sync(unsigned, bool p) {
  g_x[t_lane] = p;
  g_bar.arrive_and_wait();
  unsigned m = 0;
  for (int i = 0; i < 32; ++i) m |= (unsigned)(g_x[i] != 0) << i;
  g_bar.arrive_and_wait();
  return m;
}
inline int __ffs(unsigned m) { return __builtin_ffs((int)m); }
namespace csa2 {
inline void set_error(unsigned) {}
}
"""

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include <thread>
#include "dense_plan.cuh"
using namespace csa2;
// args: seqs n_q n_max workers uniform change_at after length...; prints "w b pair len s0 s1 whole slot" per segment
int main(int argc, char **argv) {
  DenseArgs a = {};
  a.seqs = atoi(argv[1]);
  a.n_q = atoi(argv[2]);
  a.n_max = atoi(argv[3]);
  a.workers = atoi(argv[4]);
  g_change_at = atol(argv[6]);
  g_after = atoi(argv[7]);
  std::vector<int32_t> len;
  for (int i = 8; i < argc; ++i) len.push_back(atoi(argv[i]));
  a.n_vis = atoi(argv[5]) ? nullptr : len.data();
  g_lo = len.data();
  g_hi = g_lo + len.size();
  std::vector<std::thread> warp;
  for (int lane = 0; lane < 32; ++lane)
    warp.emplace_back([&, lane] {
      t_lane = lane;
      for (int w = 0; w < a.workers; ++w) {
        int64_t total;
        int workers;
        DenseWalk k = dense_walk(a, w, lane, total, workers);
        DenseSegment g;
        while (lane == 0 && dense_next(a, w, k, g))
          printf("%d %d %d %d %d %d %d %d %d\n", w, g.b, g.pair, g.len, g.s0, g.s1, (int)g.whole, g.slot,
                 dense_worker(total, workers, 0) == 0 && dense_worker(total, workers, total) == workers - 1);
        g_bar.arrive_and_wait();
      }
    });
  for (auto &t : warp) t.join();
  return g_bad ? 3 : 0;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    shutil.copy(os.path.join(CSRC, "dense_plan.cuh"), d)
    (d / "kernels.cuh").write_text(SHIM)
    (d / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++20", "-O1", "-pthread", str(d / "main.cpp"), "-o", str(d / "plan")], check=True)

    def run(lens, n_q, n_max, workers, uniform=0, change_at=-1, after=0):
        r = subprocess.run([str(d / "plan"), *map(str, (len(lens), n_q, n_max, workers, uniform, change_at, after, *lens))],
                           capture_output=True, text=True, timeout=20)
        assert r.returncode == 0, "a length was read outside the array"
        return [tuple(map(int, x.split())) for x in r.stdout.splitlines()]
    return run


def check_split(segments, lens, n_q, workers):
    pairs = (n_q + 1) // 2
    steps = [-(-n // 256) for n in lens]
    total = pairs * sum(steps)
    used = min(total, workers)
    seen, count = {}, [0] * workers
    for w, b, pair, length, s0, s1, whole, slot, ends in segments:
        assert length == lens[b] and 0 <= pair < pairs and 0 <= s0 < s1 <= steps[b] and ends
        assert bool(whole) == (s0 == 0 and s1 == steps[b])
        assert slot in (2 * w, 2 * w + 1)
        seen.setdefault((b, pair), []).append((s0, s1, w, slot))
        count[w] += s1 - s0
    for b, n in enumerate(lens):
        for pair in range(pairs):
            parts = sorted(seen.pop((b, pair), []))
            assert (parts[0][0], parts[-1][1]) == (0, steps[b]) if n else not parts
            assert all(x[1] == y[0] and y[2] == x[2] + 1 and y[3] == 2 * y[2] for x, y in zip(parts, parts[1:]))
    assert not seen
    assert sum(count) == total and all(c in (total // used, -(-total // used)) for c in count[:used]) and not any(count[used:])


CASES = [([1], 1, 76), ([300], 1, 2), ([257, 600], 3, 12), ([1000, 0, 1], 5, 30), ([0, 0, 5, 0], 2, 4), ([513] * 40, 64, 76),
         ([(37 * i) % 301 for i in range(70)], 1, 50), ([2 ** 31 - 512], 1, 76), ([2 ** 31 - 512, 0, 2 ** 31 - 700], 4001, 76),
         ([100] * 40 + [6000, 0] + [256] * 38, 2, 76)]


@pytest.mark.parametrize("lens,n_q,workers", CASES)
def test_every_unit_is_in_one_range(plan, lens, n_q, workers):
    total = (n_q + 1) // 2 * sum(-(-n // 256) for n in lens)
    if total > 10 ** 6 and n_q > 1:   # (only the ranges' ends: the pairs are too many to print)
        n_q = 2
    check_split(plan(lens, n_q, max(lens), workers), lens, n_q, workers)


def test_random_lengths(plan):
    rng = random.Random(5)
    for _ in range(6):
        n = rng.choice([1, 7, 31, 32, 33, 64, 100])
        lens = [rng.choice([0, 1, 255, 256, 257, rng.randrange(5000)]) for _ in range(n)]
        n_q = rng.randrange(1, 9)
        workers = rng.choice([1, 5, 76])
        check_split(plan(lens, n_q, 5000, workers), lens, n_q, workers)


@pytest.mark.parametrize("n_max,seqs,n_q", [(70000, 1, 33), (500, 90, 1)])
def test_uniform_lengths(plan, n_max, seqs, n_q):
    check_split(plan([n_max] * seqs, n_q, n_max, 76, uniform=1), [n_max] * seqs, n_q, 76)


@pytest.mark.parametrize("seqs,change_at,after", [(40, 45, 0), (40, 100, 0), (100, 230, 1), (33, 40, 300), (5, 6, 0), (40, 45, 5000)])
def test_the_walk_ends_when_lengths_change(plan, seqs, change_at, after):
    """The result is undefined then, but every walk ends and stays inside the arrays."""
    lens, n_q = [900] * seqs, 3
    for w, b, pair, length, s0, s1, whole, slot, ends in plan(lens, n_q, 5000, 20, change_at=change_at, after=after):
        assert 0 <= b < seqs and 0 <= pair < 2 and 0 <= s0 < s1 <= -(-length // 256) and length <= 5000 and slot in (2 * w, 2 * w + 1)
