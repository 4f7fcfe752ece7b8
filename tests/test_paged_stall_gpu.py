"""Waits that give up inside the tensor-memory kernel: a build whose first four
key heads each have barriers that never complete (queries, free slots,
probabilities, sums).  Those heads' rows become NaN, the other heads are right,
and the GPU goes on."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
import dit_token_b200 as dit
from _paged import Batch, check_attention
for d in (64, 128, 256):
    for chunks, pasts in (([300], [3000]), ([300, 200], [500, 6000])):
        x = Batch(chunks, pasts, 10, 5, d, seed=d).fill()
        for keys in (1, max(x.kv)):  # whole key axes, and cut ones
            for _ in range(3):
                out = torch.full((x.rows, x.hq * d), 7.0, dtype=torch.bfloat16, device="cuda")
                lse = torch.full((x.rows, x.hq), 7.0, dtype=torch.float32, device="cuda")
                dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table, x.kv_lens(), x.cs, x.cp, max_kv_len=keys,
                                        max_chunk=300, out=out, lse=lse, **x.sizes())
                torch.cuda.synchronize()
                ok = x.valid()
                heads = out.view(x.rows, x.hq, d)
                assert bool(heads[ok][:, :8].isnan().all()), "a row of a head that gave up"
                assert bool((out[~ok] == 7).all()) and bool((lse[~ok] == 7).all())
                {lse}
                y = Batch(chunks, pasts, 2, 1, d, seed=d)  # the head that did not
                y.q, y.k_cache, y.v_cache, y.table = x.q[:, 8 * d:], x.k_cache[:, :, 4:], x.v_cache[:, :, 4:], x.table
                check_attention(y, heads[:, 8:].flatten(1), lse[:, 8:], True, 0)
print("went on")
"""


@pytest.fixture(scope="module")
def stalling(tmp_path_factory):
    from dit_token_b200 import build
    return build.build(out=str(tmp_path_factory.mktemp("stall") / "libdit_stall.so"), defines=["DIT_STALL=1"])


def run(lib, lse="pass"):
    code = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"), lse=lse)
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, DIT_TOKEN_LIB=lib), capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "went on" in r.stdout, r.stdout + r.stderr


def test_rows_of_a_block_that_gave_up_are_nan(stalling):
    run(stalling)


def test_so_is_their_lse(stalling):
    run(stalling, lse='assert bool(lse[ok][:, :8].isnan().all()), "lse of a row of a head that gave up"')
