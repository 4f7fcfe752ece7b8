"""Every attention kernel over a paged cache where the others are tested too:
more chunk sequences than a warp looks at in one round, mixed batches of that
size, key axes cut under a window, caches that only the warp-level kernel takes,
and sums whose every term is known."""
import pytest
import torch

import dit_token_b200 as dit
from _paged import BF16_HALF, Batch, check_attention, ints

pytestmark = pytest.mark.gpu

# a page size that the tensor-memory kernel takes, one it takes in boxes of four
# rows, and one that only the warp-level kernel does
PAGES = [16, 20, 10]


def attend(x, causal=True, window=0, lens=None, **hints):
    out = torch.full((x.rows, x.hq * x.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((x.rows, x.hq), 7.0, dtype=torch.float32, device="cuda")
    dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table, x.kv_lens() if lens is None else lens, x.cs, x.cp,
                            causal=causal, window=window, out=out, lse=lse, **x.sizes(), **hints)
    ok = x.valid()
    assert bool((out[~ok] == 7).all()) and bool((lse[~ok] == 7).all())
    return out, lse


def attend_and_check(x, causal=True, window=0, **hints):
    """Whole key axes (the smallest hint) and cut ones (the cache's capacity, the longest)."""
    for keys in (1, 0, max(x.kv)):
        out, lse = attend(x, causal, window, max_kv_len=keys, **hints)
        check_attention(x, out, lse, causal, window)


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("count", [33, 40, 150])
def test_many_chunks(count, page):
    chunks = [9 + (13 * b) % 30 for b in range(count)]
    pasts = [(97 * b) % 900 for b in range(count)]
    attend_and_check(Batch(chunks, pasts, 4, 1, 64, page=page, seed=count).fill())


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("count", [40, 90])
@pytest.mark.parametrize("d", [64, 128])
def test_many_next_tokens_beside_chunks(d, count, page):
    """Single tokens, chunks of few rows, chunks and empty sequences, more than 32
    of them, their key axes cut: two long caches among short ones."""
    chunks = [(1, 7, 1, 60, 0)[b % 5] for b in range(count)]
    pasts = [(4000 if b in (3, 36) else 31 * b % 300) for b in range(count)]
    attend_and_check(Batch(chunks, pasts, 4, 2, d, page=page, pad=4, seed=count).fill(), max_chunk=60)


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 100, 1000, 2500])
def test_a_cut_key_axis_under_a_window(window, causal, d, page):
    attend_and_check(Batch([70, 150], [3000, 2000], 4, 2, d, page=page, seed=window + d).fill(), causal, window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [33, 64, 65, 129, 300])
@pytest.mark.parametrize("hq,hk", [(2, 2), (5, 1), (40, 8)])
def test_the_warp_level_kernel(hq, hk, n, d):
    attend_and_check(Batch([n, 40], [500, 3], hq, hk, d, page=7, seed=n).fill())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_the_warp_level_kernel_where_rows_see_nothing(causal, d):
    x = Batch([40, 1, 200, 0, 90], [0, 0, 0, 0, 0], 4, 2, d, page=6, kv_lens=[25, 0, 100, 0, 0]).fill()
    attend_and_check(x, causal)


# Zero queries make every visible key's probability 1 before the division, in any
# number format, and values are whole numbers up to 3, so all sums are exact in
# fp32 (at most 3 * 5000 < 2^24).  What is left of o are a reciprocal, a product
# and a rounding: 2^-22 and half a step of bf16 of o itself; one value row read
# wrongly moves the sum by 1 or more, which is more than that wherever the sum is
# below 2^7.  lse = ln(count) to 2^-20.
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 130), (False, 1000), (True, 5)])
@pytest.mark.parametrize("chunks,pasts,hq,hk", [([1, 1, 1], [0, 1700, 4100], 4, 2), ([140, 60], [3000, 500], 4, 2),
                                                ([140, 1, 3], [300, 2600, 64], 8, 1), ([200], [1900], 3, 3)])
def test_sums_of_whole_numbers(chunks, pasts, hq, hk, causal, window, d, page):
    x = Batch(chunks, pasts, hq, hk, d, page=page, seed=d + page).fill()
    x.q[x.valid()] = 0
    g = torch.Generator(device="cuda").manual_seed(d)
    for b, n in enumerate(x.kv):
        where = x.place(b, 0, n)
        x.v_cache[where] = torch.randint(-3, 4, (n, hk, d), device="cuda", generator=g).bfloat16()
    for keys in (1, 0, max(x.kv)):
        out, lse = attend(x, causal, window, max_kv_len=keys, max_chunk=max(chunks))
        for b, n in enumerate(chunks):
            total = x.kv[b]
            j, p = torch.arange(total, device="cuda")[None], total - n + torch.arange(n, device="cuda")[:, None]
            sees = (j <= p) if causal else torch.ones(n, total, dtype=torch.bool, device="cuda")
            if window:
                sees = sees & (j > p - window)
            values = x.v_cache[x.place(b, 0, total)].double().repeat_interleave(hq // hk, 1)  # [total, hq, d]
            count = sees.sum(1).double()
            want = torch.einsum("nt,thd->nhd", sees.double(), values) / count[:, None, None]
            r = slice(x.first[b], x.first[b] + n)
            err = (out[r].double().view(n, hq, d) - want).abs()
            assert bool((err <= want.abs() * (BF16_HALF + 2.0 ** -21)).all())
            assert bool(((lse[r].double() - torch.log(count)[:, None]).abs() <= 2.0 ** -20 * 16).all())


@pytest.mark.parametrize("page", [16, 10])
def test_a_captured_mixed_batch_follows_its_lengths(page):
    """A replayed call whose lengths, tables and chunks' places have changed
    since it was captured, over a cut key axis, with its own workspace."""
    x = Batch([70, 1, 20, 1], [2000, 700, 0, 4000], 4, 2, 128, page=page, seed=page).fill()
    lens, full = x.kv_lens(), list(x.kv)
    out = torch.zeros(x.rows, x.hq * x.d, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(x.rows, x.hq, device="cuda")

    def call():
        dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table, lens, x.cs, x.cp, out=out, lse=lse, **x.sizes())
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for kv in ([70, 1, 20, 3], [1000, 701, 20, 4001], [90, 5, 20, 1], full):
        x.kv = kv
        lens.copy_(x.kv_lens())
        graph.replay()
        check_attention(x, out, lse, True, 0)
        eager, eager_lse = attend(x)
        ok = x.valid()
        assert torch.equal(out[ok], eager[ok]) and torch.equal(lse[ok], eager_lse[ok])


def test_two_chunk_calls_at_once():
    """Two streams over cut key axes, a workspace each."""
    xs = [Batch([70, 1], [6000, 3000 + i], 4, 2, 128, seed=i).fill() for i in range(2)]
    want, lens = [attend(x)[0] for x in xs], [x.kv_lens() for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    outs = [dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table, n, x.cs, x.cp, stream=s, **x.sizes())
            for _ in range(5) for x, n, s in zip(xs, lens, streams)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        ok = xs[i % 2].valid()
        assert torch.equal(o[ok], want[i % 2][ok])


def test_workspaces_at_their_exact_size():
    """What stands behind a workspace keeps its bytes, for each kind of call."""
    for chunks, page in (([1, 1], 16), ([200, 1], 16), ([300], 16), ([200, 1], 10)):
        x = Batch(chunks, [3000] * len(chunks), 4, 2, 128, page=page, seed=4).fill()
        n = dit.dit_paged_attention_workspace(x.rows, len(chunks), max_kv_len=x.max_pages * page, **x.sizes())
        buf = torch.full((n + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
        out, lse = attend(x, workspace=buf[:n])
        check_attention(x, out, lse, True, 0)
        assert n > 0 and bool((buf[n:] == 0xa5).all())
