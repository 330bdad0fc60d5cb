"""Limits of the shared-prefix plan: contexts near 2^31, and the deal of tiles to CTA pairs."""
import pytest

import paged_mla_decode_latent_gb300 as mla


@pytest.fixture(scope="module", autouse=True)
def built():
    mla.build()


@pytest.mark.parametrize("heads,dtype", [(128, mla.KV_BF16), (16, mla.KV_BF16), (8, mla.KV_FP8_E4M3)])
@pytest.mark.parametrize("batch", [1, 200])
@pytest.mark.parametrize("prefix", [0, 100, 1 << 22])
def test_own_keys_end_below_2_31(heads, dtype, batch, prefix):
    """The kernels count keys in int32: a chunk of own keys must not end past it."""
    planned = 0
    for n in (2 ** 31 - 1, 2 ** 31 - 65, 2 ** 31 - 2 ** 20, 2 ** 31 - 2 ** 26, 2 ** 30):
        try:
            p = mla.prefix_plan([n] * batch, prefix, heads, 1, 4096, dtype, False, 152)
        except mla.MLADecodeError as e:
            assert e.status == mla.ERR_UNSUPPORTED
            continue
        planned += 1
        assert p.own_chunk > 0
        assert p.prefix_len + p.own_splits * p.own_chunk < 2 ** 31
        assert p.own_splits * p.own_chunk >= n - prefix
    assert planned > 0 or batch > 1


SHARES = """
#include <cstdio>
#include "internal.h"
int main() {
  long long total; int pairs;
  while (std::scanf("%lld %d", &total, &pairs) == 2) {
    const mla::PrefixShares s(total, pairs);
    bool ok = s.start(0) == 0 && s.start(pairs) == total;
    for (int i = 0; i < pairs; ++i) {
      const long long n = s.start(i + 1) - s.start(i);
      ok = ok && n >= total / pairs && n <= (total + pairs - 1) / pairs;
      if (n > 0) ok = ok && s.pair_of(s.start(i)) == i && s.pair_of(s.start(i + 1) - 1) == i;
    }
    std::printf("%d\\n", (int)ok);
  }
}
"""


def test_shares_and_their_inverse(tmp_path):
    """Pair i's units [start(i), start(i + 1)) tile [0, total), differ by at most one in number, and
    pair_of finds each back: below the pair count, at its multiples, past 32 bits."""
    import os
    import shutil
    import subprocess
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    src, exe = tmp_path / "shares.cpp", tmp_path / "shares"
    src.write_text(SHARES)
    subprocess.run(["g++", "-std=c++17", "-w", "-I" + os.path.join(os.path.dirname(mla.__file__), "csrc"),
                    "-I" + os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
                    str(src), "-o", str(exe)], check=True)
    cases = [(t, n) for n in (1, 2, 3, 7, 76, 256)
             for t in sorted({1, 2, 5, n - 1, n, n + 1, 2 * n, 3 * n - 1, 1000, 131075, 2 ** 31, 2 ** 32 + 5, 2 ** 40 + 77})
             if t > 0]
    got = subprocess.run([str(exe)], input="".join(f"{t} {n}\n" for t, n in cases), capture_output=True,
                         text=True, check=True).stdout.split()
    assert got == ["1"] * len(cases), [c for c, g in zip(cases, got) if g != "1"]
