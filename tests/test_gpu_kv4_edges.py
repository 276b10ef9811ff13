"""The 4-bit cache and its attention in the calls that are easily forgotten:
pools past 32 bits, very many sequences, empty tables, shared pages, other
streams, several graphs, values that are not finite."""
import numpy as np
import pytest

import oracle.kv4 as o
from kv4_helpers import Batch, check_attention, random_pages, to_dev, to_host

pytestmark = pytest.mark.gpu


def queries(b, heads):
    return b.rng.standard_normal((b.n_tok, heads, b.hd)).astype(np.float32)


@pytest.mark.parametrize("n,H", [([1, 1], 4), ([9, 5], 4), ([40, 60], 4)])
def test_pool_past_32_bits(gq, n, H):
    """Pages scattered over 5 GiB: append, read and attention give what they
    give over a small pool, bit for bit."""
    import torch
    P, n_kv, hd = 64, 2, 128
    b = Batch(101, n, [150, 200], P, n_kv, hd)
    page_bytes = b.pages.shape[1]
    many = 5 * 2 ** 30 // page_bytes
    far = np.linspace(0, many - 1, len(b.pages)).astype(np.int32)[::-1]
    pool = torch.empty(many * page_bytes, dtype=torch.uint8, device="cuda")
    x = to_dev(b.rng.standard_normal((b.n_tok, H + 2 * n_kv, hd)).astype(np.float32))
    lens, q_start = b.dev()
    rope = gq.Rope(gq.gq_rope_freqs(hd, 10000.0)[0].cuda())
    got = []
    for table, pages in ((b.table, to_dev(b.pages)), (far[b.table], pool)):
        where = [int(i) for i in (far if pages is pool else range(len(b.pages)))]
        for i, page in zip(where, to_dev(b.pages)):
            pages.view(-1, page_bytes)[i].copy_(page)
        cache = gq.KV4Cache(pages.view(-1), to_dev(np.ascontiguousarray(table)), P, n_kv, hd)
        q = gq.gq_kv4_append(cache, x[:, H:H + n_kv], x[:, H + n_kv:], lens, q_start, rope=rope, q=x[:, :H])
        K, V = gq.gq_kv4_read(cache, lens, b.n_tok, q_start)
        out = gq.gq_kv4_attn(cache, q, lens, q_start, max_q=max(n))
        held = torch.stack([pages.view(-1, page_bytes)[i] for i in where])
        got.append([to_host(t) for t in (held, q, K, V, out)])
    for near, distant in zip(*got):
        assert np.array_equal(near, distant)
    assert not np.array_equal(got[0][0], b.pages)


def test_stride_past_32_bits(gq):
    # two tokens whose rows lie more than 2^31 floats apart
    import torch
    H, hd, far = 2, 64, 2 ** 31 + 192
    b = Batch(102, [2], [40], 16, 1, hd)
    q = queries(b, H)
    buf = torch.empty(far + H * hd, device="cuda")
    x = buf.as_strided((2, H, hd), (far, hd, 1))
    x.copy_(to_dev(q))
    lens, q_start = b.dev()
    pos = to_dev(np.array([3, 9], np.int32))
    rope = gq.Rope(gq.gq_rope_freqs(hd, 10000.0)[0].cuda())
    want = to_host(gq.gq_qk_rope(to_dev(q), pos, rope))
    assert np.array_equal(to_host(gq.gq_qk_rope(x, pos, rope)), want)
    check_attention(b, to_host(gq.gq_kv4_attn(b.cache(gq), x, lens, q_start)), q, hd ** -0.5, True, 0)
    gq.gq_qk_rope(x, pos, rope, out=x)
    assert np.array_equal(to_host(x.contiguous()), want)


def test_more_sequences_than_a_grid_takes(gq):
    """70 000 sequences of one kv head, on pages that they share."""
    n, hd = 70000, 32
    rng = np.random.default_rng(103)
    pages = random_pages(rng, 7, 16, 1, hd)
    lens = 1 + np.arange(n, dtype=np.int32) % 32
    table = np.stack((np.arange(n) % 7, np.arange(n) % 5), 1).astype(np.int32)
    q = rng.standard_normal((n, 1, hd)).astype(np.float32)
    cache = gq.KV4Cache(to_dev(pages), to_dev(table), 16, 1, hd)
    dq, dl = to_dev(q), to_dev(lens)
    out = to_host(gq.gq_kv4_attn(cache, dq, dl))
    K, V = gq.gq_kv4_read(cache, dl, n)
    b = Batch(103, [1], [1], 16, 1, hd, uniform=True)
    b.pages, b.table, b.lens, b.n_tok = pages, table, lens, n
    rows = [0, 1, 31, 32, 65534, 65535, 65536, 69999]
    check_attention(b, out, q, hd ** -0.5, True, 0, rows=rows)
    for t in rows:
        k, v = b.sequence(t)
        assert np.array_equal(to_host(K)[t], k[-1]) and np.array_equal(to_host(V)[t], v[-1])
    # the others: equal pages, length and query give equal bits
    again = to_host(gq.gq_kv4_attn(cache, to_dev(q[::-1].copy()), to_dev(lens[::-1].copy())))
    period = 7 * 5 * 32
    t = np.arange(n - period)
    same = to_host(gq.gq_kv4_attn(cache, to_dev(np.broadcast_to(q[:1], q.shape).copy()), dl))
    assert np.array_equal(same[t], same[t + period]) and np.isfinite(again).all()


@pytest.mark.parametrize("n", [[1, 1], [3, 40]])
def test_table_without_pages(gq, n):
    """A capacity of zero: nothing is stored, read rows stay, attention is 0."""
    import torch
    b = Batch(104, n, [50, 60], 16, 2, 64)
    x = to_dev(b.rng.standard_normal((b.n_tok, 8, 64)).astype(np.float32))
    lens, q_start = b.dev()
    pages = to_dev(b.pages)
    cache = gq.KV4Cache(pages.view(-1), torch.empty((2, 0), dtype=torch.int32, device="cuda"), 16, 2, 64)
    q = torch.full((b.n_tok, 4, 64), 2.0, device="cuda")
    gq.gq_kv4_append(cache, x[:, 4:6], x[:, 6:], lens, q_start, q=x[:, :4], q_out=q)
    assert (to_host(q) == 2.0).all() and np.array_equal(to_host(pages), b.pages)
    K = torch.full((b.n_tok, 2, 64), 3.0, device="cuda")
    gq.gq_kv4_read(cache, lens, b.n_tok, q_start, K=K)
    assert (to_host(K) == 3.0).all()
    assert not to_host(gq.gq_kv4_attn(cache, q, lens, q_start, max_q=max(n))).any()


@pytest.mark.parametrize("n,H,hd", [([1], 40, 64), ([1, 1], 64, 128), ([1], 150, 96), ([2, 1], 33, 32)])
def test_many_heads_on_one_kv_head(gq, n, H, hd):
    # more rows of one token than the kernel for few rows takes
    b = Batch(105, n, [90] + [333] * (len(n) - 1), 16, 1, hd)
    q = queries(b, H)
    lens, q_start = b.dev()
    out = gq.gq_kv4_attn(b.cache(gq), to_dev(q), lens, q_start, max_q=max(n))
    check_attention(b, to_host(out), q, hd ** -0.5, True, 0)


@pytest.mark.parametrize("n", [[1, 3], [7, 2], [50, 5]])
def test_default_bound_on_rows(gq, n):
    # without max_q every row of a ragged batch is computed
    b = Batch(106, n, [90, 60], 16, 2, 64)
    q = queries(b, 4)
    lens, q_start = b.dev()
    check_attention(b, to_host(gq.gq_kv4_attn(b.cache(gq), to_dev(q), lens, q_start)), q, 64 ** -0.5, True, 0)


@pytest.mark.parametrize("n", [[1, 1], [4, 4], [40, 33]])
def test_sequences_that_share_pages(gq, n):
    b = Batch(107, n, [130, 100], 16, 2, 64)
    b.table[1, :6] = b.table[0, :6]           # a common prefix of 96 tokens
    b.table[0, 7] = b.table[0, 6]             # and a page met twice by one sequence
    q = queries(b, 4)
    lens, q_start = b.dev()
    out = to_host(gq.gq_kv4_attn(b.cache(gq), to_dev(q), lens, q_start, max_q=max(n)))
    check_attention(b, out, q, 64 ** -0.5, True, 0)


@pytest.mark.parametrize("n", [[3, 1], [9, 6], [40, 60]])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_queries_that_are_not_finite(gq, n, bad):
    """Such a row is NaN where it sees keys, and no other row is."""
    b = Batch(108, n, [90, 160], 16, 2, 64)
    q = queries(b, 4)
    q[1, 2, 17] = bad
    lens, q_start = b.dev()
    out = to_host(gq.gq_kv4_attn(b.cache(gq), to_dev(q), lens, q_start, max_q=max(n)))
    assert np.isnan(out[1, 2]).all()
    q[1, 2] = out[1, 2] = 0.0
    want = o.attention(q[1], *o.rows(b.q_start, b.lens, b.n_tok)[1][1:], int(b.lens[0]), *b.sequence(0), 64 ** -0.5)[0]
    out[1, 2] = want[2]                       # the zeroed query's mean, so that all rows can be compared
    check_attention(b, out, q, 64 ** -0.5, True, 0)


@pytest.mark.parametrize("n", [[1], [6], [50]])
def test_attention_over_scales_of_another_writer(gq, n):
    """Scales of 11 bits: the values are rounded once to fp16."""
    b = Batch(109, n, [200], 16, 1, 64)
    pages = b.pages.reshape(len(b.pages), 2, -1)
    code = 16 * 32
    d = b.rng.standard_normal((len(pages), 2, 32)).astype(np.float16)
    pages[..., code:] = np.ascontiguousarray(d).view(np.uint8)
    q = queries(b, 2)
    lens, q_start = b.dev()
    out = to_host(gq.gq_kv4_attn(b.cache(gq), to_dev(q), lens, q_start, max_q=n[0]))
    exact = b.sequence
    b.sequence = lambda s, p=None: tuple(t.astype(np.float16).astype(np.float64) for t in exact(s, p))
    assert any((t != u).any() for t, u in zip(exact(0), b.sequence(0)))
    check_attention(b, out, q, 64 ** -0.5, True, 0)


def test_very_long_sequence(gq):
    b = Batch(110, [1, 2], [300001, 70], 1024, 1, 64)
    q = queries(b, 2)
    lens, q_start = b.dev()
    out = to_host(gq.gq_kv4_attn(b.cache(gq), to_dev(q), lens, q_start, max_q=2))
    check_attention(b, out, q, 64 ** -0.5, True, 0)
    out = to_host(gq.gq_kv4_attn(b.cache(gq), to_dev(q), lens, q_start, max_q=2, window=70001))
    check_attention(b, out, q, 64 ** -0.5, True, 70001)


def test_results_belong_to_the_given_stream(gq):
    """A result made on another stream does not take memory that work still
    queued on the current one may be reading."""
    import torch
    b = Batch(111, [1, 1], [40, 50], 16, 2, 64, uniform=True)
    s = torch.cuda.Stream()
    cache, (lens, _) = b.cache(gq), b.dev()
    x = to_dev(b.rng.standard_normal((2, 8, 64)).astype(np.float32))
    pos = to_dev(np.array([1, 2], np.int32))
    rope = gq.Rope(torch.ones(32, device="cuda"))
    torch.cuda.synchronize()
    calls = (lambda: [gq.gq_qk_rope(x[:, :4], pos, rope, stream=s)],
             lambda: [gq.gq_kv4_append(cache, x[:, 4:6], x[:, 6:], lens, rope=rope, q=x[:, :4], stream=s)],
             lambda: list(gq.gq_kv4_read(cache, lens, 2, stream=s)),
             lambda: [gq.gq_kv4_attn(cache, x[:, :4], lens, stream=s)])
    for call in calls:
        for heads in (2, 4):
            gone = torch.empty((2, heads, 64), device="cuda")
            at = gone.data_ptr()
            del gone                          # the current stream's allocator has it again
            again = torch.empty((2, heads, 64), device="cuda").data_ptr()
            assert again == at
            made = call()
            s.synchronize()
            assert all(t.data_ptr() != at for t in made)


def test_two_graphs_at_once(gq):
    """Two captured layers with workspaces of their own, replayed side by side
    with other lengths, eager calls between."""
    import torch
    H, n_kv, hd, P = 8, 2, 128, 64
    rope = gq.Rope(gq.gq_rope_freqs(hd, 10000.0)[0].cuda())
    layers = []
    for i in range(2):
        b = Batch(112 + i, [1, 1], [4000, 900], P, n_kv, hd, uniform=True)
        cache, (lens, _) = b.cache(gq), b.dev()
        x = to_dev(b.rng.standard_normal((2, H + 2 * n_kv, hd)).astype(np.float32))
        ws = torch.empty(gq.gq_kv4_attn_ws_bytes(cache, H, 1, cache.capacity), dtype=torch.uint8, device="cuda")
        assert ws.numel() > 0

        def step(ws, x=x, cache=cache, lens=lens):
            q = gq.gq_kv4_append(cache, x[:, H:H + n_kv], x[:, H + n_kv:], lens, rope=rope, q=x[:, :H])
            return gq.gq_kv4_attn(cache, q, lens, workspace=ws)

        step(ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(ws)
        layers.append((step, lens, graph, out, torch.cuda.Stream()))
    for turn in range(5):
        for step, lens, *_ in layers:
            lens.copy_(to_dev(np.array([4000 - 700 * turn, 901 + turn], np.int32)))
        torch.cuda.synchronize()
        for _, _, graph, _, stream in layers:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for step, _, _, out, _ in layers:
            assert np.array_equal(to_host(out), to_host(step(None))), turn


@pytest.mark.parametrize("n,H,n_kv,hd", [
    ([1] * 40 + [150, 0, 0, 2] + [1] * 30 + [33, 1], 4, 2, 64),      # more sequences than one search step takes
    ([0, 128, 0, 32, 33, 1, 0], 8, 2, 128),                          # tiles that end where a sequence does
    ([31, 1, 64, 95, 1], 4, 1, 256),
    ([0] * 200 + [40] + [0] * 200, 2, 2, 32),
])
def test_prompts_and_single_tokens_in_one_batch(gq, n, H, n_kv, hd):
    """Row tiles dealt to sequences of very different lengths; rows before the
    first and behind the last sequence are left as they were."""
    import torch
    lens = [m + (17 * i) % 90 for i, m in enumerate(n)]
    b = Batch(114, n, lens, 16, n_kv, hd)
    q = queries(b, H)
    lens, q_start = b.dev()
    for max_q in (None, max(n)):
        full = torch.full((b.n_tok + 8, H, hd), 6.0, device="cuda")
        out = full.clone()
        full[5:-3] = to_dev(q)
        gq.gq_kv4_attn(b.cache(gq), full, lens, q_start + 5, max_q=max_q, out=out)
        got = to_host(out)
        assert (got[:5] == 6.0).all() and (got[-3:] == 6.0).all()
        check_attention(b, got[5:-3], q, hd ** -0.5, True, 0)


def test_attention_with_offsets_that_are_none(gq):
    """Offsets that descend or leave the rows: nothing outside the arrays is
    touched, and sequences before the first such offset are computed (but for
    rows that a later one claims too)."""
    import torch
    b = Batch(115, [40, 3, 100], [40, 3, 100], 32, 2, 96)
    q = queries(b, 4)
    cache, dq = b.cache(gq), to_dev(q)
    lens, q_start = b.dev()
    want = to_host(gq.gq_kv4_attn(cache, dq, lens, q_start, max_q=100))
    for bad in ([0, 40, 30, 143], [-5, 40, 43, 143], [0, 40, 43, 999], [2147483647] * 4, [-2147483648] * 4,
                [0, 2147483647, -2147483648, 143]):
        guard = torch.full((b.n_tok + 2, 4, 96), 9.0, device="cuda")
        gq.gq_kv4_attn(cache, dq, lens, to_dev(np.array(bad, np.int32)), max_q=100, out=guard[1:-1])
        got = to_host(guard)
        assert (got[0] == 9.0).all() and (got[-1] == 9.0).all()
        if bad[:2] == [0, 40]:
            own = min(40, bad[2])
            assert np.array_equal(got[1:1 + own], want[:own])


@pytest.mark.parametrize("n", [[1, 1], [6, 3], [50, 3]])
@pytest.mark.parametrize("window", [1, 40, 700, 3000, 8999, 9000])
def test_windows_over_long_sequences(gq, n, window):
    # cut into the parts that the window's keys call for
    b = Batch(116, n, [9000, 2500], 64, 1, 64)
    q = queries(b, 4)
    lens, q_start = b.dev()
    for causal in (True, False):
        out = gq.gq_kv4_attn(b.cache(gq), to_dev(q), lens, q_start, max_q=max(n), causal=causal, window=window)
        check_attention(b, to_host(out), q, 64 ** -0.5, causal, window)


def test_prompts_and_single_tokens_as_two_calls(gq):
    """The sequences of each kind by slices of the same arrays, into one output."""
    import torch
    n = [1] * 6 + [70, 41]
    b = Batch(117, n, [700, 1, 33, 64, 2000, 90, 100, 300], 16, 2, 128)
    q = queries(b, 8)
    lens, q_start = b.dev()
    whole, dq = b.cache(gq), to_dev(q)
    out = torch.full(q.shape, 4.0, device="cuda")
    for lo, hi, max_q in ((0, 6, 1), (6, 8, 70)):
        cache = gq.KV4Cache(whole.pages, whole.table[lo:hi], 16, 2, 128)
        gq.gq_kv4_attn(cache, dq, lens[lo:hi], q_start[lo:hi + 1], max_q=max_q, out=out)
        if lo == 0:
            assert (to_host(out)[6:] == 4.0).all()
    check_attention(b, to_host(out), q, 128 ** -0.5, True, 0)


@pytest.mark.parametrize("n,lens,H,n_kv,hd", [
    ([2100], [2100], 2, 1, 64),
    ([2100, 33], [2100, 1500], 4, 2, 128),
    ([1, 1, 1, 1, 1], [9000, 0, 576, 577, 1], 4, 2, 64),
    ([5, 8, 3], [9000, 20, 700], 4, 1, 256),
])
def test_lengths_far_under_the_bound(gq, n, lens, H, n_kv, hd):
    """Parts without keys: sequences and rows with few keys under a bound that
    others reach, and under one far above every length."""
    b = Batch(118, n, lens, 64, n_kv, hd)
    b.table = np.concatenate((b.table, np.full((len(n), 600), -1, np.int32)), 1)
    q = queries(b, H)
    dev_lens, q_start = b.dev()
    rows = None if b.n_tok < 20 else [0, 1, 31, 32, 255, 256, 383, 384, 576, 577, 1000, 2047, 2099] + list(range(2100, b.n_tok))
    for max_len in (max(lens), b.table.shape[1] * 64):
        for causal in (True, False):
            out = gq.gq_kv4_attn(b.cache(gq), to_dev(q), dev_lens, q_start, max_q=max(n), max_len=max_len, causal=causal)
            check_attention(b, to_host(out), q, hd ** -0.5, causal, 0, rows=rows)
