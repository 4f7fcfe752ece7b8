"""The attention over a paged cache where its kernels have to agree with one
another: malformed packings over a cut key axis."""
import math

import pytest
import torch

import dit_token_b200 as dit
from _paged import Batch, check_attention, ints

pytestmark = pytest.mark.gpu


def attend(x, cs, cp, rows, causal=True, window=0, **hints):
    """dit_paged_attention over the first ``rows`` rows of the batch's buffer
    with a packing of the test's own.  Outputs start as 7 and the workspace as
    finite rubbish, so that what was not computed is seen."""
    out = torch.full((x.rows, x.hq * x.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((x.rows, x.hq), 7.0, dtype=torch.float32, device="cuda")
    hints.setdefault("max_chunk", max(x.chunks))
    hints.setdefault("max_kv_len", max(x.kv))
    nbytes = dit.dit_paged_attention_workspace(rows, len(x.chunks), **x.sizes(), **hints)
    work = torch.full((nbytes,), 0x3f, dtype=torch.uint8, device="cuda")
    dit.dit_paged_attention(x.q[:rows], x.k_cache, x.v_cache, x.table, x.kv_lens(), cs, cp, causal=causal,
                            window=window, out=out[:rows], lse=lse[:rows], workspace=work, **x.sizes(), **hints)
    return out, lse


# Chunks and lengths whose key axis is cut, in pages that the tensor-memory
# kernel takes (16) and that only the warp-level one does (10); more sequences
# than a warp looks at in one round; a single token among the chunks.
CUT = [([60, 300], [5000, 4000], 2), ([1, 60, 300], [700, 5000, 4000], 2), ([20] * 40, [2200] * 40, 1)]


@pytest.mark.parametrize("page", [16, 10])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("chunks,pasts,hk", CUT)
def test_a_sequence_past_the_buffer_is_skipped_whole(chunks, pasts, hk, d, page):
    """The last sequence's final rows lie behind the buffer: none of its rows
    is written, the others are as if it were not there."""
    x = Batch(chunks, pasts, 2 * hk, hk, d, page=page, slack=0, seed=d + page).fill()
    rows = x.first[-2] + chunks[-1] - 3
    out, lse = attend(x, x.cs, x.cp, rows)
    last = x.first[-2]
    assert bool((out[last:] == 7).all()) and bool((lse[last:] == 7).all())
    x.chunks = chunks[:-1] + [0]
    check_attention(x, out, lse, True, 0)
    assert bool((out[~x.valid()] == 7).all()) and bool((lse[~x.valid()] == 7).all())


@pytest.mark.parametrize("page", [16, 10])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("slot", [8, 24])
def test_a_slot_shorter_than_its_chunk(slot, d, page):
    """A sequence of 40 valid rows in a padded slot of fewer: those that have a
    padded row are its chunk, whichever kernel they fall to beside a chunk of
    300 whose key axis is cut."""
    x = Batch([slot, 300], [4000, 4000], 4, 2, d, page=page, slack=40, seed=slot + d).fill()
    out, lse = attend(x, ints([0, 40, 340]), x.cp, x.rows, max_chunk=400)
    check_attention(x, out, lse, True, 0)
    assert bool((out[~x.valid()] == 7).all()) and bool((lse[~x.valid()] == 7).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("sign", [1, -1])
def test_maxima_that_grow_at_every_step(d, sign):
    """Every step of 128 keys tops the ones before it by more than the running
    maximum may lag (2^8), for some rows (and falls for others, whose queries
    are negative), so probabilities are computed against an old maximum first
    and then again: 30 calls agree bit for bit and with the definition."""
    x = Batch([300], [2500], 4, 2, d, seed=d).fill()
    where = x.place(0, 0, x.kv[0])
    step = (torch.arange(x.kv[0], device="cuda") // 128).float()
    # 20 per step in the exponent's powers of two; the noise in the keys stays
    x.k_cache[where] = (x.k_cache[where].float() + (step * 14.0)[:, None, None] / d ** 0.5).bfloat16()
    x.q[:300] = 1.0
    x.q[1:300:3] = -1.0
    x.q[:300] *= sign
    first = None
    for keys in [0] * 10 + [1] * 10 + [max(x.kv)] * 10:  # cut and whole key axes
        out, lse = attend(x, x.cs, x.cp, x.rows, max_kv_len=keys or x.max_pages * x.page)
        if first is None or keys != first[2]:
            check_attention(x, out, lse, True, 0)
            first = (out, lse, keys)
        assert torch.equal(out[x.valid()], first[0][x.valid()]) and torch.equal(lse[x.valid()], first[1][x.valid()])


@pytest.mark.parametrize("page", [16, 10])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 50, 127, 128, 129, 700])
def test_tokens_behind_every_window_may_hold_anything(window, causal, d, page):
    """A token that no query of its sequence's chunk sees (its page may have
    been given away) is NaN in the cache or has no page at all: the outputs are
    those over the other tokens, whole key axes and cut ones, chunks and single
    tokens."""
    chunks, pasts = [140, 1, 33], [1500, 900, 2100]
    x = Batch(chunks, pasts, 4, 2, d, page=page, seed=window).fill()
    want, expired = x.table.clone(), [max(0, p - window + 1) for p in pasts]
    for b, n in enumerate(expired):
        where = x.place(b, 0, n)
        x.k_cache[where], x.v_cache[where] = math.nan, math.nan
        x.table[b, :n // page // 2] = -7
    outs = [attend(x, x.cs, x.cp, x.rows, causal, window, max_kv_len=keys)
            for keys in (1, max(x.kv), x.max_pages * page)]
    x.table = want
    for b, n in enumerate(expired):  # the definition multiplies them by 0 as well: finite for it
        where = x.place(b, 0, n)
        x.k_cache[where], x.v_cache[where] = 0.0, 0.0
    for out, lse in outs:
        check_attention(x, out, lse, causal, window)
