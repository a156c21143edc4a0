"""The check of adapter descriptors, in a CPU build of the function that the kernels call:
no offset, however large, passes for a place inside the packs."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

I64_MAX = (1 << 63) - 1

SOURCE = r'''
#include "desc.hpp"
extern "C" bool check(int64_t a_off, int64_t b_off, int32_t rank, int32_t max_rank, int64_t d_in,
                      int64_t d_out, int64_t a_elems, int64_t b_elems) {
  return lora::desc_ok(lora_adapter_desc{a_off, b_off, rank, 1.f}, max_rank, d_in, d_out, a_elems, b_elems);
}
'''


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    from rl_lora_linear_amd import build as B
    d = tmp_path_factory.mktemp("desc")
    src, lib = os.path.join(d, "check.hip"), os.path.join(d, "check.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([B.HIPCC, *B.CFLAGS, "--offload-host-only", "-shared", src, "-o", lib], check=True, capture_output=True)
    fn = ctypes.CDLL(lib).check
    fn.restype, fn.argtypes = ctypes.c_bool, [ctypes.c_int64] * 2 + [ctypes.c_int32] * 2 + [ctypes.c_int64] * 4
    return fn


def _want(a, b, r, max_rank, d_in, d_out, a_elems, b_elems):
    """The rule in whole numbers of any size."""
    return (8 <= r <= 64 and r % 8 == 0 and r <= max_rank and a >= 0 and b >= 0 and a % 8 == 0 and b % 8 == 0 and
            a + r * d_in <= a_elems and b + r * d_out <= b_elems)


def test_offsets_near_the_largest_integer(check):
    for big in (I64_MAX - 7, I64_MAX - 15, I64_MAX - 16 * 128 - 7, (1 << 62), I64_MAX - I64_MAX % 8 - 64 * (1 << 20)):
        for elems in (0, 4096, 1 << 40, I64_MAX):
            for a, b in ((big, 0), (0, big), (big, big)):
                for d in (64, 128, 1 << 20):
                    args = (a, b, 16, 64, d, d, elems, elems)
                    assert check(*args) == _want(*args), args
    assert not check(I64_MAX - 7, 0, 16, 64, 128, 64, 4096, 4096)
    assert not check(0, I64_MAX - 7, 16, 64, 128, 64, 4096, 4096)


def test_every_rule_at_its_border(check):
    rng = np.random.default_rng(0)
    d_in, d_out, hits = 128, 64, 0
    for _ in range(4000):
        r = int(rng.choice([-8, 0, 4, 8, 12, 16, 24, 32, 64, 72]))
        end_a, end_b = (int(v) for v in rng.choice([0, 8, 64, 4096], 2))
        a, b = (int(e + v) for e, v in zip((end_a, end_b), rng.choice([-16, -8, -1, 0, 1, 8], 2)))
        args = (a, b, r, int(rng.choice([16, 32, 64])), d_in, d_out, end_a + max(r, 0) * d_in, end_b + max(r, 0) * d_out)
        assert check(*args) == _want(*args), args
        hits += check(*args)
    assert hits > 100
