"""How a tile of the gated recurrence looks back over the flags of the tiles before it, on the host with made-up flags: whether a
run on the GPU steps over more than one window of 64 depends on its timing."""
import subprocess

from gated_delta_rule_47_amd import _build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "kda_gated_scan.h"

// The nearest final place with flags behind it all along, by the definition; -1: none yet.
static int nearest(const std::vector<int>& f) {
  for (int p = (int)f.size() - 1; p >= 0 && f[p]; --p)
    if (f[p] == 2) return p;
  return -1;
}
struct Run {
  int got, reads, pauses;
};
// read_hook before every window, pause_hook in every pause; reads past `most` mean that it would not end.
template <typename R, typename P> static Run look(std::vector<int>& f, R read_hook, P pause_hook, int most) {
  Run r = {0, 0, 0};
  const int last = (int)f.size() - 1;
  r.got = kda::scan_look_back(
      last,
      [&](int at) {
        if (++r.reads > most) printf("does not end\n"), exit(1);
        read_hook(at == last);
        kda::ScanFlags w = {0, 0};
        for (int l = 0; l < 64; ++l) {
          const int flag = at - l >= 0 ? f[at - l] : 0;
          w.any |= (unsigned long long)(flag >= 1) << l;
          w.final |= (unsigned long long)(flag == 2) << l;
        }
        return w;
      },
      [&] { ++r.pauses, pause_hook(r.pauses); });
  return r;
}
#define CHECK(x) if (!(x)) return printf("line %d, %d places: got %d, %d reads, %d pauses\n", __LINE__, n, r.got, r.reads, r.pauses), 1

int main() {
  const auto none = [](auto) {};
  std::mt19937 g(1);
  for (int n : {1, 2, 63, 64, 65, 127, 128, 129, 200, 512, 1000}) {
    {  // the first place alone is final: windows without a pause, each once
      std::vector<int> f(n, 1);
      f[0] = 2;
      const Run r = look(f, none, none, 100);
      CHECK(r.got == 0 && r.reads == (n + 63) / 64 && r.pauses == 0);
    }
    for (int k = 0; k < n; k += 1 + n / 40) {  // one final place anywhere, some in front of it not even ready
      std::vector<int> f(n, 1);
      for (int p = 0; p < k; p += 3) f[p] = 0;
      f[k] = 2;
      const Run r = look(f, none, none, 100);
      CHECK(r.got == k && r.reads == (n - 1 - k) / 64 + 1 && r.pauses == 0);
    }
    for (int gap = 1; gap < n; gap += 1 + n / 40) {  // a place without a flag, in any window: it waits, from the newest place again
      std::vector<int> f(n, 1);
      f[0] = 2, f[gap] = 0;
      const Run r = look(f, none, [&](int i) { if (i == 3) f[gap] = 1; }, 1000);
      CHECK(r.got == 0 && r.pauses == 3 && r.reads == 3 * ((n - 1 - gap) / 64 + 1) + (n + 63) / 64);
      f[gap] = 0;
      // a place behind the gap finishes while it waits: the gap no longer matters
      if (gap + 1 < n) {
        const Run r = look(f, none, [&](int i) { if (i == 2) f[gap + 1] = 2; }, 1000);
        CHECK(r.got == gap + 1 && r.pauses == 2);
      }
    }
    {  // nothing is final until the first place is
      std::vector<int> f(n, 1);
      f[0] = 0;
      const Run r = look(f, none, [&](int i) { if (i == 4) f[0] = 2; }, 1000);
      CHECK(r.got == 0 && r.pauses == 4);
    }
    for (int k = 0; k < 300; ++k) {  // flags in any order while it looks: each goes from 0 to 1 to 2, place 0 to 2 at once
      std::vector<int> f(n);
      for (int& x : f) x = g() % 8 ? 1 : g() % 3;
      f[0] = f[0] ? 2 : 0;
      int known = -1;
      const Run r = look(f, [&](bool starts) {
        for (int i = 0; i < 1 + n / 64; ++i) {
          int& x = f[g() % n];
          if (g() % 4 == 0 && x < 2) ++x;
          if (&x == &f[0] && x == 1) x = 2;
        }
        if (starts) known = nearest(f);
      }, none, 1000000);
      CHECK(r.got >= 0 && f[r.got] == 2 && r.got >= known);
      for (int p = r.got + 1; p < n; ++p) CHECK(f[p]);
    }
  }
  printf("ok\n");
}
"""


def test_look_back_over_windows(tmp_path):
    src, prog = tmp_path / "look.hip", tmp_path / "look"
    src.write_text(PROGRAM)
    subprocess.run([_build.HIPCC, "--offload-host-only", "-O1", "-std=c++17", "-I", _build.CSRC, str(src), "-o", str(prog)],
                   check=True, capture_output=True)
    out = subprocess.run([str(prog)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout
