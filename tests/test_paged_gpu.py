"""The paged-cache operators on the GPU against their 64-bit definitions:
lengths from none to long, odd sizes, strides, layouts, masks that leave a row
empty, slots and pages that must not be read or written."""
import math

import pytest
import torch

import dit_token_b200 as dit
from _paged import (Batch, check_attention, check_rotation, cumulative, ints, reference_attention,
                    reference_rotation)

pytestmark = pytest.mark.gpu
NAN = math.nan

def attend(x, causal=True, window=0, hints=True, lse=True, **kw):
    """dit_paged_attention on a batch, with canaries around what it may write."""
    buf = torch.full((x.rows, x.hq * x.d + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, 16:16 + x.hq * x.d]
    ls = torch.full((x.rows, x.hq), 7.0, dtype=torch.float32, device="cuda") if lse else None
    if hints:
        kw.setdefault("max_chunk", max(x.chunks))
        kw.setdefault("max_kv_len", max(x.kv))
    got = dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table, x.kv_lens(), x.cs, x.cp, causal=causal,
                                  window=window, out=out, lse=ls, **x.sizes(), **kw)
    assert got.data_ptr() == out.data_ptr()
    assert bool((buf[:, :16] == 7).all()) and bool((buf[:, 16 + x.hq * x.d:] == 7).all())
    assert bool((out[~x.valid()] == 7).all()), "a padding row was written"
    if lse:
        assert bool((ls[~x.valid()] == 7).all()), "a padding row of lse was written"
    return out, ls


def attend_and_check(x, causal=True, window=0, **kw):
    out, lse = attend(x, causal, window, **kw)
    check_attention(x, out, lse, causal, window)
    return out, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 193, 1000, 5000])
def test_one_token(d, kv):
    attend_and_check(Batch([1], [kv - 1], 4, 2, d, seed=kv).fill())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [2, 7, 16, 17, 33, 64, 65, 127, 128, 129, 257, 300])
def test_one_chunk_behind_a_prefix(d, n):
    attend_and_check(Batch([n], [n % 5 * 37], 4, 2, d, page=24, seed=n).fill())


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (5, 1), (8, 1), (6, 2), (40, 8), (17, 1), (64, 2), (130, 1)])
@pytest.mark.parametrize("n", [1, 3, 70])
def test_head_groups(hq, hk, n):
    attend_and_check(Batch([n, n], [100, 5], hq, hk, 64, seed=hq).fill())


@pytest.mark.parametrize("page", [1, 7, 10, 12, 16, 20, 100, 256])
@pytest.mark.parametrize("chunks,pasts", [([1, 1, 1], [0, 99, 255]), ([130, 1, 40], [70, 256, 0])])
def test_page_sizes(page, chunks, pasts):
    attend_and_check(Batch(chunks, pasts, 4, 2, 128, page=page, seed=page).fill())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 2, 63, 64, 65, 200, 100000])
@pytest.mark.parametrize("chunks,pasts", [([1, 1], [300, 20]), ([150, 3], [200, 400])])
def test_masks(d, causal, window, chunks, pasts):
    attend_and_check(Batch(chunks, pasts, 4, 2, d, seed=window).fill(), causal, window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(d, causal):
    """kv_lens below the chunk's length (a caller's mistake, or nothing
    cached): causal rows before the first key see nothing; 0 keys, no row."""
    x = Batch([40, 1, 200, 0, 9], [0, 0, 0, 0, 0], 4, 2, d, kv_lens=[25, 0, 100, 0, 9]).fill()
    out, lse = attend_and_check(x, causal)
    first = x.first[1]
    assert bool((out[first] == 0).all()) and bool((lse[first] == -math.inf).all())
    if causal:
        assert bool((out[:15] == 0).all()) and bool((lse[:15] == -math.inf).all())
        assert bool((lse[15:40] > -math.inf).all())


def test_ragged_batch_with_empty_sequences():
    chunks = [0, 1, 300, 0, 1, 17, 128, 0]
    attend_and_check(Batch(chunks, [10, 900, 55, 0, 0, 1000, 128, 3], 8, 2, 128, seed=5).fill())


def test_many_sequences():
    """More sequences than a warp scans at once."""
    chunks = [(7 * b) % 5 for b in range(150)]
    pasts = [(13 * b) % 200 for b in range(150)]
    attend_and_check(Batch(chunks, pasts, 4, 4, 64, pad=1, seed=6).fill())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 90])
def test_hints_never_change_what_is_computed(d, n):
    x = Batch([n, 1], [3000, 700], 4, 2, d, seed=8).fill()
    for hints in (dict(), dict(max_chunk=1, max_kv_len=1), dict(max_chunk=1, max_kv_len=64),
                  dict(max_chunk=10**9, max_kv_len=10**12), dict(max_kv_len=2000)):
        attend_and_check(x, hints=False, **hints)


@pytest.mark.parametrize("n,past", [(1, 20000), (50, 9000), (300, 3000)])
def test_long_caches(n, past):
    for causal in (True, False):
        attend_and_check(Batch([n], [past], 8, 2, 128, page=64, seed=n).fill(), causal)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_extreme_scores(d):
    """Scores of several hundred: the running maximum moves by more than the
    exponent range, and the softmax is nearly one key."""
    for n, past in ((1, 700), (150, 300)):
        attend_and_check(Batch([n], [past], 2, 1, d, scale=6.0, seed=d).fill(scale=6.0))
    # rising scores: every key tops the ones before it
    x = Batch([130], [500], 2, 1, d, seed=1).fill()
    where = x.place(0, 0, x.kv[0])
    x.q[:130] = 1.0
    x.k_cache[where] = (torch.arange(x.kv[0], device="cuda") / 16.0)[:, None, None].expand(-1, 1, d).bfloat16()
    attend_and_check(x)
    x.k_cache[where] = x.k_cache[where].neg()
    attend_and_check(x)


def test_head_major_cache_and_softmax_scale():
    x = Batch([70, 1], [90, 500], 8, 2, 128, hnd=True, seed=9).fill()
    assert not x.k_cache.is_contiguous()
    out, lse = attend(x, softmax_scale=0.03)
    check_attention(x, out, lse, True, 0, scale=0.03)
    attend_and_check(x)


def test_without_lse_and_with_allocated_output():
    x = Batch([70, 1], [90, 500], 8, 2, 128, seed=10).fill()
    out, _ = attend(x)
    plain = dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table, x.kv_lens(), x.cs, x.cp, **x.sizes())
    assert plain.shape == (x.rows, x.hq * x.d)
    check_attention(x, plain, None, True, 0)


@pytest.mark.parametrize("n", [1, 200])
def test_pages_outside_the_cache_read_as_zeros(n):
    for bad in (-1, -2**31, 10**6, 2**31 - 1):
        x = Batch([n], [400], 4, 2, 128, seed=11).fill()
        dead = x.table_host[0][3]
        out, lse = attend(x)
        x.table[0, 3] = bad
        out, lse = attend(x)
        x.table[0, 3] = dead  # the definition looks the page up, and puts zeros there
        check_attention(x, out, lse, True, 0, dead_pages=(dead,))


def test_lengths_past_the_table_stop_at_its_end():
    x = Batch([1], [63], 4, 2, 128, page=16, seed=12).fill()
    table = x.table[:, :4].contiguous()
    out = dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, table, ints([70]), x.cs, x.cp, **x.sizes())
    x.q[1:] = 0
    ref, _, size, _ = reference_attention(x, True, 0)  # the 64 tokens that the table names
    assert float((out.double().view_as(ref)[0] - ref[0]).abs().max()) <= float((2.0**-7 * size[0]).max())


def test_malformed_packing_is_skipped():
    x = Batch([5, 6], [40, 50], 4, 2, 64, slack=0, seed=13).fill()
    out = torch.full((x.rows, x.hq * x.d), 7.0, dtype=torch.bfloat16, device="cuda")
    for cs, cp in (([0, 5, 11], [0, 8, 10**6]), ([0, 5, 11], [0, x.rows - 2, x.rows + 90]), ([0, 5, 11], [-8, 8, 16]),
                   ([0, 10**6, 10**6 + 4], [0, 8, 16])):
        dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table, x.kv_lens(), ints(cs), ints(cp), out=out,
                                **x.sizes())
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """A cache of more than 2^31 elements: pages at both its ends."""
    hk, d, page = 8, 128, 64
    pages = (1 << 31) // (page * hk * d) + 40
    caches = [torch.empty(pages, page, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    x = Batch([130, 1], [70, 200], 16, hk, d, page=page, seed=14)
    far = [pages - 1 - i for i in range(6)]
    x.table = ints([[far[0], 3, far[1], far[2], 9], [far[3], 1, far[4], 0, far[5]]])
    x.k_cache, x.v_cache = caches
    x.fill()
    attend_and_check(x)
    freqs, _ = dit.dit_rope_frequencies(64)
    before = [x.k_cache[far[3]].clone(), x.v_cache[1].clone()]
    dit.dit_qkv_rope_append(x.q, x.k, x.v, x.k_cache, x.v_cache, x.table, ints([70, 200]), x.cs, x.cp, freqs=freqs,
                            q_out=torch.empty_like(x.q), **x.sizes())
    where = x.place(0, 70, 200)
    assert torch.equal(x.v_cache[where].flatten(1), x.v[:130])
    assert torch.equal(x.k_cache[far[3]], before[0]) and torch.equal(x.v_cache[1], before[1])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hk", [(8, 2), (40, 1)])
def test_next_tokens_beside_chunks(d, hq, hk):
    """A mixed batch: chunks, chunks of few rows and single tokens, with long
    caches and without, more key tiles than blocks and fewer."""
    chunks = [1, 300, 1, 8, 9, 1, 0, 33, 2]
    pasts = [9000, 500, 0, 700, 64, 4000, 10, 0, 2500]
    x = Batch(chunks, pasts, hq, hk, d, seed=d).fill()
    for causal, window in ((True, 0), (False, 0), (True, 300)):
        attend_and_check(x, causal, window)


def test_caches_of_other_strides():
    """Keys and values in one tensor, heads of a wider cache, pages with slack
    between them (whose stride is no multiple of a slot's), heads apart from
    both: what TMA can follow and what it cannot."""
    for n in (1, 150):
        for make in ("one tensor", "wider heads", "slack", "loose heads"):
            x = Batch([n, 2], [200, 70], 4, 2, 128, page=32, seed=22)
            pages, page, hk, d = x.k_cache.shape
            if make == "one tensor":
                both = torch.full((pages, 2, page, hk, d), NAN, dtype=torch.bfloat16, device="cuda")
                x.k_cache, x.v_cache = both[:, 0], both[:, 1]
            else:
                size, strides = {
                    "wider heads": (page * (hk + 3) * d, (page * (hk + 3) * d, (hk + 3) * d, d, 1)),
                    "slack": (page * hk * d + 8, (page * hk * d + 8, hk * d, d, 1)),
                    "loose heads": (page * hk * d * 3, (page * hk * d * 3, d + 8, page * (d + 8) + 16, 1)),
                }[make]
                x.k_cache, x.v_cache = (torch.full((pages * size,), NAN, dtype=torch.bfloat16, device="cuda").as_strided(
                    (pages, page, hk, d), strides) for _ in range(2))
            x.fill()
            attend_and_check(x)
            freqs, _ = dit.dit_rope_frequencies(64)
            v = x.v.clone()
            dit.dit_qkv_rope_append(x.q, x.k, x.v, x.k_cache, x.v_cache, x.table, ints(x.pasts), x.cs, x.cp, freqs=freqs,
                                    q_out=torch.empty_like(x.q), **x.sizes())
            assert torch.equal(x.v_cache[x.place(0, 200, 200 + n)].flatten(1), v[:n])
            attend_and_check(x)


def test_captured_without_a_workspace():
    """The workspace and the output come from the graph's own pool."""
    x = Batch([1, 200], [3000, 500], 8, 2, 128, seed=23).fill()
    want, _ = attend(x, hints=False)
    lens = x.kv_lens()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table, lens, x.cs, x.cp, **x.sizes())
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out[x.valid()], want[x.valid()])


@pytest.mark.parametrize("n", [1, 260])
def test_repeats_bit_for_bit_and_in_a_graph(n):
    """Two calls agree; a captured call follows the lengths it finds at replay."""
    x = Batch([n, 1], [900, 40], 8, 2, 128, seed=15).fill()
    a, la = attend(x)
    b, lb = attend(x)
    assert torch.equal(a, b) and torch.equal(la[x.valid()], lb[x.valid()])
    out, lse = torch.zeros_like(a), torch.zeros_like(la)
    lens = x.kv_lens()
    nbytes = dit.dit_paged_attention_workspace(x.rows, 2, max_chunk=n, max_kv_len=max(x.kv), **x.sizes())
    work = torch.empty(nbytes, dtype=torch.uint8, device="cuda")

    def call():
        dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table, lens, x.cs, x.cp, max_chunk=n, max_kv_len=max(x.kv),
                                out=out, lse=lse, workspace=work, **x.sizes())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    full = list(x.kv)
    for kv in ([full[0] - 500, 3], [n, 41], full):
        x.kv = [max(kv[0], n), kv[1]]
        lens.copy_(x.kv_lens())
        graph.replay()
        check_attention(x, out, lse, True, 0)
    assert torch.equal(out[x.valid()], a[x.valid()])


def test_on_another_stream():
    x = Batch([1, 1], [3000, 2000], 8, 2, 128, seed=16).fill()
    a, _ = attend(x, hints=False)  # the same call, so the same bits
    lens = x.kv_lens()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table, lens, x.cs, x.cp, stream=s, **x.sizes())
            for s in (side, side.cuda_stream, side)]
    side.synchronize()
    for o in outs:
        assert torch.equal(o[x.valid()], a[x.valid()])


def test_two_calls_at_once():
    """Two streams, a workspace each."""
    xs = [Batch([1, 1], [30000, 20000 + i], 8, 2, 128, page=64, seed=17 + i).fill() for i in range(2)]
    want, lens = [attend(x)[0] for x in xs], [x.kv_lens() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = []
    for _ in range(5):
        for x, n, s in zip(xs, lens, streams):
            outs.append(dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table, n, x.cs, x.cp, stream=s,
                                                max_chunk=1, max_kv_len=max(x.kv), **x.sizes()))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o[xs[i % 2].valid()], want[i % 2][xs[i % 2].valid()])


# ------------------------------------------------------------ rotation

STARTS = [0, 5, 100_000, -3, 2**31 - 200]


def rotation_case(mode, rotary, d, hq, hk, norm, grid, seed=0, chunks=(3, 0, 17, 1, 40)):
    x = Batch(list(chunks), [0] * len(chunks), hq, hk, d, seed=seed)
    freqs, gain = dit.dit_rope_frequencies(rotary, scaling="yarn", factor=8.0, original_len=512)
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(freqs=freqs, attn_scale=gain, rope_mode=mode)
    ref = dict(rotary=rotary, mode=mode, freqs=freqs, gain=float(torch.tensor(gain)), starts=STARTS[:len(chunks)])
    if norm:
        kw["q_weight"] = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16()
        kw["k_weight"] = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16()
    if grid:
        grids = [(2, 2, 3), (4, 5, 6), (60, 40, 50), (0, 4, 4), (3, 2, 2)][:len(chunks)]
        side = rotary // 3 // 2 * 2
        sections = (rotary - 2 * side, side, side)
        table = torch.cat([dit.dit_rope_frequencies(n, theta=500.0)[0] for n in sections if n])
        kw.update(rope_grid=ints([list(v) for v in grids]), grid_freqs=table, sections=sections)
        ref.update(grids=grids, grid_freqs=table, sections=sections)
    return x, kw, ref


@pytest.mark.parametrize("mode", ["interleaved", "half"])
@pytest.mark.parametrize("d,rotary", [(64, 64), (64, 8), (64, 40), (128, 128), (128, 64), (128, 120), (128, 16),
                                      (256, 256), (256, 72)])
@pytest.mark.parametrize("norm,grid", [(True, False), (False, False), (True, True), (False, True)])
def test_rotation(mode, d, rotary, norm, grid):
    x, kw, ref = rotation_case(mode, rotary, d, 5, 3, norm, grid, seed=rotary)
    q_out = torch.full((x.rows, 5 * d), 7.0, dtype=torch.bfloat16, device="cuda")
    k_out = torch.full((x.rows, 3 * d), 7.0, dtype=torch.bfloat16, device="cuda")
    dit.dit_qk_rope_scaled(x.q, x.k, x.cs, x.cp, num_q_heads=5, num_k_heads=3, head_dim=d, pos_offset=ints(STARTS),
                           q_out=q_out, k_out=k_out, **kw)
    ok = x.valid()
    for t, out, heads, w in ((x.q, q_out, 5, "q_weight"), (x.k, k_out, 3, "k_weight")):
        want, size = reference_rotation(t, x.chunks, x.first, heads, d, weight=kw.get(w), **ref)
        check_rotation(out[ok], want[ok], size[ok], w)
        assert bool((out[~ok] == 7).all())
        if not norm and rotary < d:  # what does not turn passes bit for bit
            assert torch.equal(out.view(x.rows, heads, d)[ok][..., rotary:], t.reshape(x.rows, heads, d)[ok][..., rotary:])
    # in place gives the same bits
    q, k = x.q.clone(), x.k.clone()
    dit.dit_qk_rope_scaled(q, k, x.cs, x.cp, num_q_heads=5, num_k_heads=3, head_dim=d, pos_offset=ints(STARTS), **kw)
    assert torch.equal(q[ok], q_out[ok]) and torch.equal(k[ok], k_out[ok]) and bool(q[~ok].isnan().all())


@pytest.mark.parametrize("hq,hk", [(0, 3), (3, 0), (1, 1), (40, 8), (9, 33)])
@pytest.mark.parametrize("chunks", [(1, 1, 1), (700, 1, 2500)])
def test_rotation_head_counts(hq, hk, chunks):
    x, kw, ref = rotation_case("half", 64, 64, max(hq, 1), max(hk, 1), True, False, chunks=chunks)
    ref["starts"] = [0, 0, 0]
    q = x.q[:, :hq * 64] if hq else torch.empty(x.rows, 0, dtype=torch.bfloat16, device="cuda")
    dit.dit_qk_rope_scaled(q, x.k[:, :hk * 64], x.cs, x.cp, num_q_heads=hq, num_k_heads=hk, head_dim=64,
                           q_out=(qo := torch.zeros(x.rows, hq * 64, dtype=torch.bfloat16, device="cuda")),
                           k_out=(ko := torch.zeros(x.rows, hk * 64, dtype=torch.bfloat16, device="cuda")), **kw)
    ok = x.valid()
    for t, out, heads, w in ((x.q, qo, hq, "q_weight"), (x.k, ko, hk, "k_weight")):
        if heads:
            want, size = reference_rotation(t, x.chunks, x.first, heads, 64, weight=kw[w], **ref)
            check_rotation(out[ok], want[ok], size[ok], w)


@pytest.mark.parametrize("norm", [True, False])
def test_no_rotation(norm):
    x, kw, ref = rotation_case("none", 64, 128, 3, 2, norm, False)
    kw["freqs"] = None
    q, k = x.q.clone(), x.k.clone()
    dit.dit_qk_rope_scaled(q, k, x.cs, x.cp, num_q_heads=3, num_k_heads=2, head_dim=128, **kw)
    ok = x.valid()
    if not norm:
        assert torch.equal(q[ok], x.q[ok]) and torch.equal(k[ok], x.k[ok])
    else:
        want, size = reference_rotation(x.q, x.chunks, x.first, 3, 128, weight=kw["q_weight"], **ref)
        check_rotation(q[ok], want[ok], size[ok])


def test_agrees_with_the_unscaled_operator():
    """Unscaled tables over whole heads are what dit_qk_rmsnorm_rope turns by:
    both are within their roundings of one value, two bf16 steps apart at most."""
    x, kw, _ = rotation_case("interleaved", 128, 128, 4, 2, True, False)
    freqs, gain = dit.dit_rope_frequencies(128)
    kw.update(freqs=freqs, attn_scale=gain)
    a, b = (x.q.clone(), x.k.clone()), (x.q.clone(), x.k.clone())
    dit.dit_qk_rope_scaled(*a, x.cs, x.cp, num_q_heads=4, num_k_heads=2, head_dim=128, pos_offset=ints(STARTS), **kw)
    dit.dit_qk_rmsnorm_rope(*b, kw["q_weight"], kw["k_weight"], x.cs, x.cp, num_q_heads=4, num_k_heads=2,
                            head_dim=128, pos_offset=ints(STARTS))
    ok = x.valid()
    for s, t in zip(a, b):
        s, t = s[ok].float(), t[ok].float()
        assert bool(((s - t).abs() <= 2.0**-7 * t.abs() + 2.0**-16).all())


# ------------------------------------------------------------ append

@pytest.mark.parametrize("mode", ["interleaved", "half", "none"])
@pytest.mark.parametrize("d,rotary,page,hnd", [(64, 32, 7, False), (128, 128, 16, True), (256, 64, 100, False)])
@pytest.mark.parametrize("chunks,pasts", [([1, 1, 1], [0, 15, 300]), ([5, 0, 37, 200], [3, 9, 0, 111])])
def test_append(mode, d, rotary, page, hnd, chunks, pasts):
    for norm, grid in ((False, False), (True, mode != "none")):
        x = Batch(chunks, pasts, 6, 2, d, page=page, hnd=hnd, seed=rotary)
        _, kw, ref = rotation_case(mode, rotary, d, 6, 2, norm, grid, chunks=chunks)
        ref["starts"] = pasts
        before = x.k_cache.clone(), x.v_cache.clone()
        q_out = torch.full((x.rows, 6 * d), 7.0, dtype=torch.bfloat16, device="cuda")
        k, v = x.k.clone(), x.v.clone()
        dit.dit_qkv_rope_append(x.q, x.k, x.v, x.k_cache, x.v_cache, x.table, ints(pasts), x.cs, x.cp, q_out=q_out,
                                **kw, **x.sizes())
        ok = x.valid()
        want, size = reference_rotation(x.q, x.chunks, x.first, 6, d, weight=kw.get("q_weight"), **ref)
        check_rotation(q_out[ok], want[ok], size[ok], "q")
        assert bool((q_out[~ok] == 7).all())
        assert torch.equal(x.k.view(torch.int16), k.view(torch.int16))
        assert torch.equal(x.v.view(torch.int16), v.view(torch.int16))
        want, size = reference_rotation(x.k, x.chunks, x.first, 2, d, weight=kw.get("k_weight"), **ref)
        touched = torch.zeros(x.k_cache.shape[:2], dtype=torch.bool, device="cuda")
        for b, n in enumerate(chunks):
            where = x.place(b, pasts[b], pasts[b] + n)
            r = slice(x.first[b], x.first[b] + n)
            check_rotation(x.k_cache[where], want[r], size[r], "k")
            assert torch.equal(x.v_cache[where].flatten(1), x.v[r])
            touched[where] = True
        for now, then in zip((x.k_cache, x.v_cache), before):  # every other slot keeps its bits
            assert torch.equal(now[~touched].view(torch.int16), then[~touched].view(torch.int16))


def test_append_positions_apart_from_slots():
    """pos_offset moves the angles and leaves the slots."""
    x = Batch([9], [20], 2, 2, 64, seed=3)
    freqs, gain = dit.dit_rope_frequencies(64)
    dit.dit_qkv_rope_append(x.q, x.k, x.v, x.k_cache, x.v_cache, x.table, ints([20]), x.cs, x.cp, freqs=freqs,
                            pos_offset=ints([7000]), **x.sizes())
    want, size = reference_rotation(x.k, x.chunks, x.first, 2, 64, rotary=64, mode="interleaved", freqs=freqs, gain=1.0,
                                    starts=[7000])
    check_rotation(x.k_cache[x.place(0, 20, 29)], want[:9], size[:9])


@pytest.mark.parametrize("bad", [-1, -2**31, 10**6, 2**31 - 1])
def test_append_drops_tokens_without_a_page(bad):
    x = Batch([40, 8], [3, 0], 2, 2, 64, page=16)
    x.table[0, 1] = bad  # tokens 16 .. 31 of the first sequence
    before = x.v_cache.clone()
    freqs, _ = dit.dit_rope_frequencies(64)
    # the second sequence claims to be past its table's end
    dit.dit_qkv_rope_append(x.q, x.k, x.v, x.k_cache, x.v_cache, x.table, ints([3, 2**31 - 4]), x.cs, x.cp,
                            freqs=freqs, **x.sizes())
    kept = torch.zeros(x.k_cache.shape[:2], dtype=torch.bool, device="cuda")
    for first, last, row in ((3, 16, 0), (32, 43, 29)):
        where = x.place(0, first, last)
        kept[where] = True
        assert torch.equal(x.v_cache[where].flatten(1), x.v[row:row + last - first])
    assert torch.equal(x.v_cache[~kept].view(torch.int16), before[~kept].view(torch.int16))


def test_one_sequence_twice_in_a_batch():
    """Two sequences that share a prefix's pages (read only) and own their last one."""
    x = Batch([1, 1], [32, 32], 4, 2, 128, page=16, seed=21).fill()
    x.table[1, :2] = x.table[0, :2]
    attend_and_check(x)


# ------------------------------------------------------------ as they are used

@pytest.mark.parametrize("d,hq,hk,causal,window", [(128, 8, 2, True, 0), (64, 4, 4, False, 0), (128, 4, 1, False, 150),
                                                   (256, 2, 2, True, 90)])
def test_a_stream_of_chunks_and_tokens(d, hq, hk, causal, window):
    """Chunks, then single tokens, each appended and attended: every step's
    output is the softmax over all keys so far, computed in 64 bits from the
    rows themselves (their keys and values as the cache holds them)."""
    steps = [[50, 7], [130, 0], [1, 1], [1, 64], [1, 1]]
    pasts = [0, 0]
    x = Batch([max(s[b] for s in steps) for b in range(2)], [200, 200], hq, hk, d, page=24, seed=d)
    freqs, gain = dit.dit_rope_frequencies(d // 2, scaling="ntk", factor=4.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    wq, wk = ((1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16() for _ in range(2))
    lens = ints(pasts)
    for chunks in steps:
        x.chunks, x.first = chunks, cumulative([-(-n // 8) * 8 for n in chunks])
        x.cs, x.cp = ints(cumulative(chunks)), ints(x.first)
        raw = torch.randn(x.rows, (hq + 2 * hk) * d, device="cuda", generator=g).bfloat16()
        q, k, v = raw.split([hq * d, hk * d, hk * d], 1)
        x.q = dit.dit_qkv_rope_append(q, k, v, x.k_cache, x.v_cache, x.table, lens, x.cs, x.cp, freqs=freqs,
                                      attn_scale=gain, q_weight=wq, k_weight=wk, rope_mode="half", **x.sizes())
        ref = dict(rotary=d // 2, mode="half", freqs=freqs, gain=gain, starts=pasts)
        want, size = reference_rotation(k, chunks, x.first, hk, d, weight=wk, **ref)
        for b, n in enumerate(chunks):
            where = x.place(b, pasts[b], pasts[b] + n)
            r = slice(x.first[b], x.first[b] + n)
            check_rotation(x.k_cache[where], want[r], size[r], "k")
            assert torch.equal(x.v_cache[where].flatten(1), v[r])
        pasts = [a + n for a, n in zip(pasts, chunks)]
        lens = ints(pasts)
        x.kv = list(pasts)
        out, lse = attend(x, causal, window)
        check_attention(x, out, lse, causal, window)


def test_refusals_with_tensors():
    x = Batch([3], [5], 4, 2, 64).fill()
    freqs, _ = dit.dit_rope_frequencies(64)
    args = (x.q, x.k_cache, x.v_cache, x.table, x.kv_lens(), x.cs, x.cp)
    with pytest.raises(ValueError):
        dit.dit_paged_attention(*args, num_q_heads=2, num_kv_heads=2, head_dim=64)
    with pytest.raises(ValueError):
        dit.dit_paged_attention(x.q, x.k_cache, x.v_cache[:1], *args[3:], **x.sizes())
    with pytest.raises(TypeError):
        dit.dit_paged_attention(x.q, x.k_cache, x.v_cache, x.table.long(), *args[4:], **x.sizes())
    with pytest.raises(TypeError):
        dit.dit_paged_attention(*args, lse=torch.zeros(x.rows, 4, device="cuda").half(), **x.sizes())
    with pytest.raises(dit.DitError):
        dit.dit_paged_attention(*args, softmax_scale=-1.0, **x.sizes())
    with pytest.raises(ValueError):
        dit.dit_paged_attention(x.q.cpu(), *args[1:], **x.sizes())
    with pytest.raises(ValueError):
        dit.dit_qk_rope_scaled(x.q, x.k, x.cs, x.cp, num_q_heads=4, num_k_heads=2, head_dim=64, freqs=freqs,
                               q_weight=torch.ones(64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        dit.dit_qk_rope_scaled(x.q, x.k, x.cs, x.cp, num_q_heads=4, num_k_heads=2, head_dim=64, freqs=freqs.float())
    with pytest.raises(TypeError):
        dit.dit_qkv_rope_append(x.q, x.k, x.v, x.k_cache, x.v_cache, x.table, x.kv_lens()[:0], x.cs, x.cp, freqs=freqs,
                                **x.sizes())
    for window in (-1, 2**31, 2**32):
        with pytest.raises(ValueError):
            dit.dit_paged_attention(*args, window=window, **x.sizes())
    long = Batch([1], [30000], 8, 1, 64, page=64).fill()
    with pytest.raises(dit.DitError):
        dit.dit_paged_attention(long.q, long.k_cache, long.v_cache, long.table, long.kv_lens(), long.cs, long.cp,
                                workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), **long.sizes())
