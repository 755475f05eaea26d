"""Plans of a step over drafted tokens: what their workspace holds (host only)."""
import pytest

import split_kv_flash_decode_gb300 as fd
from split_kv_flash_decode_gb300 import build


@pytest.fixture(scope="module", autouse=True)
def built_lib():
    build.build()
    return fd.lib()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype,most", [("f16", 64), ("f16_e4m3kv", 64), ("f16_e2m1kv", 64), ("bf16_e2m1kv", 64), ("bf16", 32)])
def test_long_runs_have_sums_in_the_workspace(dtype, most, d):
    """A softmax group adds up to `most` tiles of 128 tokens; it takes every tile of two row tiles, every other one of one."""
    def workspace(L, n, sms=1, B=1):
        return fd.fd_tree_plan(B, 8, 2, d, [L] * B, [n] * B, 0, dtype, sms).info["workspace_bytes"]
    sums = 2 * 128 * d * 4                              # of a CTA: two groups of 128 rows
    assert workspace(2 * most * 128, 32) == 0           # 128 query rows
    assert workspace(2 * most * 128 + 1, 32) == sums
    assert workspace(most * 128, 33) == 0               # 132
    assert workspace(most * 128 + 1, 33) == sums
    assert workspace(5000 * 128, 33) == sums
    # Runs that are short although the sequence is long: records alone.
    record = 2 * 4 * 128 * (d + 2)
    assert workspace(2 * most * 128 * 10, 1, 152) == 152 * record
    assert workspace(2 * most * 128 * 10, 1, 3) == 3 * (record + sums)
    # Many sequences, none of them long.
    assert workspace(2 * most * 128, 32, 2, 40) == 0
