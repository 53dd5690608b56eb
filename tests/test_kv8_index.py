"""Index arithmetic of the 8-bit cache's kernels (csrc/kv8_index.h) at token
counts near 2^31, compiled with the host compiler and compared with 64-bit
integers.  (Signed overflow wraps there as it does on the device.)"""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "attention_attn_fwd_gb300", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None,
                                reason="no host C++ compiler")

HEAD = r"""
#include <algorithm>
#include <cstdio>
#include "kv8_index.h"
using namespace attn::kv8;
using ll = long long;
ll bad = 0, n = 0;
unsigned long long st = 88172645463325252ull;
ll rnd(ll lo, ll hi) {  // lo .. hi
  st ^= st << 13; st ^= st >> 7; st ^= st << 17;
  return lo + static_cast<ll>(st % static_cast<unsigned long long>(hi - lo + 1));
}
const ll kMost = 0x7fffffffLL - (1 << 16) - 1;  // largest capacity
"""
TAIL = r"""
  std::printf("%lld checked, %lld wrong\n", n, bad);
  return bad != 0;
}
"""


def run(tmp_path, body):
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text(HEAD + body + TAIL)
    subprocess.run(["g++", "-O2", "-fwrapv", "-std=c++17", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr


def test_append_never_leaves_the_sequence(tmp_path):
    """Every block the grid counts to, for few new tokens of many rows given:
    one that holds new tokens, or none."""
    run(tmp_path, r"""
int main() {
  auto check = [&](ll cap, ll len, ll n_new, ll Sq, ll block) {
    const ll start = len - n_new;
    const ll units = (Sq + block - 2) / block + 1;
    auto one = [&](ll u) {
      if (u < 0 || u >= units) return;
      ++n;
      const ll blk = start / block + u;
      const ll want = blk * block < len ? blk : -1;
      const ll got = append_block(static_cast<int>(start),
                                  static_cast<int>(len),
                                  static_cast<int>(block),
                                  static_cast<int>(u));
      if (got != want) {
        if (bad < 5)
          std::printf("cap %lld len %lld new %lld Sq %lld block %lld unit %lld: "
                      "%lld\n", cap, len, n_new, Sq, block, u, got);
        ++bad;
      }
    };
    const ll end = (len - 1) / block - start / block;
    for (ll u = 0; u < 4; ++u) one(u);
    for (ll u = end - 3; u < end + 4; ++u) one(u);
    for (ll u = units - 4; u < units; ++u) one(u);
    // Where a place of the block passes 2^31 and 2^32.
    for (ll p : {1ll << 31, 1ll << 32})
      for (ll u = p / block - start / block - 2; u < p / block - start / block + 3; ++u)
        one(u);
    for (int i = 0; i < 20; ++i) one(rnd(0, units - 1));
  };
  for (ll block : {16, 32, 64, 128}) {
    for (ll cap : {kMost, kMost - 1, kMost - 127, 1ll << 30, (1ll << 30) + 5, 1000ll})
      for (ll Sq : {1ll, 2ll, 65535ll, 65536ll, 70000ll, 1ll << 20, cap})
        for (ll len : {cap, cap - 1, cap - 300, cap / 2 + 1})
          for (ll n_new : {1ll, 2ll, 17ll, 300ll})
            if (Sq <= cap && n_new <= std::min(Sq, len))
              check(cap, len, n_new, Sq, block);
    for (int i = 0; i < 20000; ++i) {
      const ll cap = rnd(1, kMost), len = rnd(1, cap), Sq = rnd(1, cap);
      check(cap, len, rnd(1, std::min(len, Sq)), Sq, block);
    }
  }
""")


def test_moved_weights_reach_every_place(tmp_path):
    """Rounds and cleared places of an eviction into a cache of up to the
    largest capacity, and in place."""
    run(tmp_path, r"""
int main() {
  auto check = [&](ll cap, ll kept, ll threads, bool in_place) {
    const ll ranks = in_place ? 8 : (cap - 1) / (4 * threads) + 1;
    const ll step = 4 * threads * ranks;
    const ll want = (kept + step - 1) / step;
    const ll got = round_count(static_cast<int>(kept), static_cast<int>(step));
    ll wrong = got != want;
    for (ll rank : {0ll, 1ll, ranks / 2, ranks - 1})
      for (ll t : {0ll, threads - 1}) {
        if (rank < 0 || rank >= ranks) continue;
        const ll place = cleared_place(
            static_cast<int>(kept), static_cast<int>(rank),
            static_cast<int>(threads), static_cast<int>(t));
        wrong += place != kept + rank * threads + t;
      }
    ++n;
    if (wrong != 0 && bad++ < 5)
      std::printf("cap %lld kept %lld threads %lld: %lld rounds of %lld\n",
                  cap, kept, threads, got, want);
  };
  for (ll threads : {32, 64, 128, 256, 512})
    for (bool in_place : {false, true}) {
      for (ll cap : {kMost, kMost - 1, (1ll << 30) - 1, 1ll << 30, 5000ll, 1ll})
        for (ll kept : {cap, cap - 1, cap / 2, 1ll, 0ll})
          check(cap, kept, threads, in_place);
      for (int i = 0; i < 50000; ++i) {
        const ll cap = rnd(1, kMost);
        check(cap, rnd(0, cap), threads, in_place);
      }
    }
""")
