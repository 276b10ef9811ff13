"""Attention over the 4-bit cache against the 64-bit oracle on the GPU, with
error bounds derived in kv4_helpers.attention_bound."""
import numpy as np
import pytest

from kv4_helpers import Batch, check_attention, to_dev, to_host

pytestmark = pytest.mark.gpu


def run(gq, b, q, max_q=None, max_len=None, scale=None, causal=True, window=0, **kw):
    lens, q_start = b.dev()
    return gq.gq_kv4_attn(b.cache(gq), to_dev(q), lens, q_start, max_q=max(b.n) if max_q is None else max_q,
                          max_len=max_len, scale=scale, causal=causal, window=window, **kw)


def queries(b, heads, size=1.0):
    return (size * b.rng.standard_normal((b.n_tok, heads, b.hd))).astype(np.float32)


@pytest.mark.parametrize("n,lens,P,H,n_kv,hd,causal,window", [
    # single tokens: group sizes 1, 3, 4, 7, 8, 16 and 20, every head size
    ([1], [1], 16, 2, 2, 64, True, 0),
    ([1, 1], [15, 333], 16, 14, 2, 64, True, 0),
    ([1], [2000], 64, 8, 2, 128, True, 0),
    ([1, 1, 1], [17, 32, 700], 32, 9, 3, 96, True, 0),
    ([1, 1], [129, 64], 128, 8, 1, 256, True, 0),
    ([1], [257], 1024, 16, 1, 128, True, 0),
    ([1], [90], 16, 20, 1, 64, True, 0),
    ([1, 1], [40, 41], 16, 3, 1, 32, True, 0),
    ([1], [50], 16, 2, 1, 160, True, 0),
    ([1], [50], 16, 2, 2, 192, True, 0),
    ([1], [50], 16, 2, 1, 224, True, 0),
    # a few tokens a sequence
    ([2, 0, 3], [100, 7, 3], 16, 4, 2, 64, True, 0),
    ([4], [500], 32, 8, 2, 128, True, 0),
    ([3, 2], [40, 90], 16, 4, 2, 96, False, 0),
    # 17 to 32 rows of a sequence and kv head, and one more
    ([8], [500], 32, 8, 2, 128, True, 0),
    ([3, 1, 0], [90, 17, 0], 16, 14, 2, 64, True, 0),
    ([6, 2], [100, 7], 16, 10, 2, 256, True, 0),
    ([5, 4], [60, 333], 16, 8, 2, 96, True, 21),
    ([32], [70], 16, 2, 2, 128, False, 0),
    ([33], [70], 16, 2, 2, 128, False, 0),
    # prompts: whole, chunks, ragged, odd
    ([33], [33], 16, 2, 1, 64, True, 0),
    ([100, 65, 1], [100, 200, 70], 16, 4, 2, 128, True, 0),
    ([64], [700], 64, 8, 2, 128, True, 0),
    ([37], [37], 32, 6, 2, 96, True, 0),
    ([45], [130], 16, 4, 2, 256, True, 0),
    ([40], [77], 16, 5, 1, 32, True, 0),
    ([35], [60], 16, 3, 1, 160, True, 0),
    ([130], [130], 16, 2, 2, 64, False, 0),
    # windows: of one key, inside a tile, of several tiles, wider than everything
    ([1, 1], [300, 20], 16, 4, 2, 64, True, 1),
    ([1, 1], [300, 20], 16, 4, 2, 64, True, 50),
    ([90], [200], 16, 4, 2, 64, True, 33),
    ([90], [200], 16, 4, 2, 128, True, 1),
    ([90], [200], 16, 4, 2, 128, True, 100000),
    ([70], [300], 16, 2, 1, 128, False, 40),
])
def test_against_oracle(gq, n, lens, P, H, n_kv, hd, causal, window):
    print(f"[kv4] attn n={n} lens={lens} P={P} H={H}/{n_kv} hd={hd} causal={causal} window={window}", flush=True)
    b = Batch(sum(n) + hd + H, n, lens, P, n_kv, hd)
    q = queries(b, H)
    out = to_host(run(gq, b, q, causal=causal, window=window))
    worst = check_attention(b, out, q, hd ** -0.5, causal, window)
    print(f"[kv4] {worst:.3f} of the bound", flush=True)


@pytest.mark.parametrize("n,lens", [([1], [9000]), ([1, 1, 1], [5000, 1, 3001]), ([3], [4097]), ([7, 5], [4097, 900]),
                                    ([64], [4500])])
def test_long_contexts(gq, n, lens):
    # long enough to be cut into parts, with several lengths under one bound
    b = Batch(sum(lens), n, lens, 64, 2, 128)
    q = queries(b, 8)
    rows = None if b.n_tok < 13 else [0, 1, 31, 32, 63]
    for max_len in (max(lens), b.table.shape[1] * 64):
        out = to_host(run(gq, b, q, max_len=max_len))
        check_attention(b, out, q, 128 ** -0.5, True, 0, rows=rows)


@pytest.mark.parametrize("size", [1e-6, 1e-3, 30.0, 1e4])
@pytest.mark.parametrize("n", [[1], [40]])
def test_magnitudes_of_queries(gq, n, size):
    # nearly equal weights, sharp ones, and scores far past where exp overflows
    b = Batch(77, n, [200], 16, 2, 64)
    q = queries(b, 4, size)
    q[:, 1, ::7] *= 1e-5                      # a head with a wide range
    out = to_host(run(gq, b, q))
    check_attention(b, out, q, 64 ** -0.5, True, 0)


def test_scale_and_zero_queries(gq):
    b = Batch(78, [1, 30], [60, 60], 16, 1, 64)
    q = queries(b, 2)
    q[::3] = 0.0                              # equal weights: the mean of the values
    for scale in (0.0, 1.0, -0.3):
        out = to_host(run(gq, b, q, scale=scale))
        check_attention(b, out, q, scale, True, 0)


def test_rows_that_see_nothing_and_rows_of_none(gq):
    """Lengths of zero, more rows than cached tokens, rows behind the last
    sequence and rows past max_q."""
    import torch
    b = Batch(79, [1, 4, 2, 40], [1, 4, 9, 40], 16, 1, 64)
    b.lens[:] = [0, 2, 9, 13]
    q = queries(b, 2)
    q = np.concatenate((q, np.ones((3, 2, 64), np.float32)))
    for max_q in (40, 3):
        out = torch.full(q.shape, 5.0, device="cuda")
        lens, q_start = b.dev()
        gq.gq_kv4_attn(b.cache(gq), to_dev(q), lens, q_start, max_q=max_q, out=out)
        got = to_host(out)
        assert (got[b.n_tok:] == 5.0).all()
        assert not got[0].any() and not got[1:3].any()           # sequence 1's rows are at -2, -1, 0, 1
        rows = [3, 5, 6] + ([4] if max_q > 3 else [])
        if max_q == 40:
            assert not got[7:7 + 27].any()                        # 40 rows over 13 tokens
            rows += list(range(7 + 27, 47))
        else:
            assert (got[4] == 5.0).all() and (got[10:47] == 5.0).all()
        check_attention(b, got, q[:b.n_tok], 64 ** -0.5, True, 0, rows=rows)


@pytest.mark.parametrize("n", [[1, 1], [3, 2], [9, 10], [40, 37]])
def test_nan_in_unwritten_slots(gq, n):
    """Slots past the length hold NaN scales; so do spare pages."""
    b = Batch(80, n, [50, 37], 16, 2, 64)
    clean = b.pages.copy()
    P, part = 16, 16 * 36
    used = {(int(b.table[s, j // P]), j % P) for s in range(2) for j in range(int(b.lens[s]))}
    for page in range(len(b.pages)):
        for slot in range(P):
            if (page, slot) not in used:
                for head_kv in range(4):
                    at = head_kv * part
                    b.pages[page, at + slot * 32: at + slot * 32 + 32] = 0xFF
                    for blk in range(2):
                        o = at + 512 + 2 * (blk * P + slot)
                        b.pages[page, o: o + 2] = 0xFF
    q = queries(b, 4)
    out = to_host(run(gq, b, q))
    check_attention(b, out, q, 64 ** -0.5, True, 0, pages=clean)


@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("bits", [0x7E00, 0x7C00])
@pytest.mark.parametrize("n,lens,window", [([6], [50], 0), ([12], [50], 0), ([60], [60], 0), ([60], [130], 20), ([2], [100], 9)])
def test_nan_in_a_seen_key_reaches_only_rows_that_see_it(gq, n, lens, window, kv, bits):
    b = Batch(81, n, lens, 16, 1, 64)
    clean = b.pages.copy()
    at = lens[0] - n[0] // 2 - 1                                  # among the rows' own positions
    page, slot = int(b.table[0, at // 16]), at % 16
    o = kv * 16 * 36 + 512 + 2 * (16 + slot)                      # block 1's scale
    b.pages[page, o: o + 2] = [bits & 255, bits >> 8]
    code = kv * 16 * 36 + slot * 32 + 16
    b.pages[page, code: code + 16] = 0x99                         # no zero codes: an infinite scale gives infinities
    q = queries(b, 2)
    out = to_host(run(gq, b, q, window=window))
    pos = lens[0] - n[0] + np.arange(n[0])
    sees = (pos >= at) & ((window == 0) | (at > pos - window))
    assert np.isfinite(out[~sees]).all() and sees.any() and (n[0] == 2 or (~sees).any())   # two rows: both see it
    b.pages, poisoned = clean, b.pages
    check_attention(b, out, q, 64 ** -0.5, True, window, rows=list(np.flatnonzero(~sees)))
    b.pages = poisoned
    if bits == 0x7E00:
        assert (~np.isfinite(out[sees][..., 32:])).all()          # the block's channels (or the weights) are NaN
    else:
        assert (~np.isfinite(out[sees][..., 32:])).any()


@pytest.mark.parametrize("n", [[1], [5], [15], [50]])
def test_page_numbers_that_are_none(gq, n):
    # pages 1 and 2 of the sequence: NaN for the rows that see them, no fault
    b = Batch(82, n, [60], 16, 2, 64)
    b.table[0, 1], b.table[0, 2] = 1 << 30, -1
    q = queries(b, 4)
    out = to_host(run(gq, b, q))
    sees = 60 - n[0] + np.arange(n[0]) >= 16
    assert np.isnan(out[sees]).all()
    check_attention(b, out, q, 64 ** -0.5, True, 0, rows=list(np.flatnonzero(~sees)))
    # behind a window nothing of them is seen
    out = to_host(run(gq, b, q, window=5))
    rows = [t for t in range(n[0]) if 60 - n[0] + t - 5 + 1 >= 48 or 60 - n[0] + t < 16]
    check_attention(b, out, q, 64 ** -0.5, True, 5, rows=rows)
    # entries past the length are not looked at
    b = Batch(83, n, [60], 16, 2, 64)
    b.table = np.concatenate((b.table, np.full((1, 3), 1 << 30, np.int32)), 1)
    out = to_host(run(gq, b, q))
    check_attention(b, out, q, 64 ** -0.5, True, 0)


def test_strided_queries_and_output(gq):
    import torch
    b = Batch(84, [1, 70], [30, 100], 16, 2, 64)
    full = (b.rng.standard_normal((b.n_tok, 8, 64))).astype(np.float32)
    dev = to_dev(full)
    out = torch.full((b.n_tok, 6, 64), 3.0, device="cuda")
    lens, q_start = b.dev()
    gq.gq_kv4_attn(b.cache(gq), dev[:, 2:6], lens, q_start, max_q=70, out=out[:, 1:5])
    got = to_host(out)
    assert (got[:, 0] == 3.0).all() and (got[:, 5] == 3.0).all()
    check_attention(b, got[:, 1:5], full[:, 2:6], 64 ** -0.5, True, 0)


def test_unaligned_queries(gq):
    # four-byte aligned tensors: one float into a larger buffer
    import torch
    b = Batch(85, [1, 20], [30, 100], 16, 2, 64)
    q = queries(b, 4)
    buf = torch.zeros(q.size + 1, device="cuda")
    buf[1:] = to_dev(q).flatten()
    obuf = torch.zeros(q.size + 1, device="cuda")
    lens, q_start = b.dev()
    gq.gq_kv4_attn(b.cache(gq), buf[1:].view(q.shape), lens, q_start, max_q=20, out=obuf[1:].view(q.shape))
    check_attention(b, to_host(obuf)[1:].reshape(q.shape), q, 64 ** -0.5, True, 0)


def test_same_bits_again_and_alone(gq):
    """Two calls give the same bits, and so does a sequence in another batch
    with the same bounds."""
    b = Batch(86, [1, 1, 1], [3000, 40, 700], 64, 2, 128, uniform=True)
    q = queries(b, 8)
    first = to_host(run(gq, b, q, max_q=1))
    assert np.array_equal(first, to_host(run(gq, b, q, max_q=1)))


def test_two_streams_at_once(gq):
    # two calls in flight with a workspace each
    import torch
    b = Batch(87, [1], [9000], 64, 2, 128)
    q = queries(b, 8)
    want = to_host(run(gq, b, q))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    cache = b.cache(gq)
    lens, q_start = b.dev()
    dq = to_dev(q)
    torch.cuda.synchronize()
    outs = []
    for i in range(6):
        s = (s1, s2)[i % 2]
        out = torch.empty_like(dq)
        s.wait_stream(torch.cuda.current_stream())
        outs.append(gq.gq_kv4_attn(cache, dq, lens, q_start, out=out, stream=s))
    torch.cuda.synchronize()
    for out in outs:
        assert np.array_equal(to_host(out), want)


@pytest.mark.parametrize("n,cap", [([1, 1], 4096), ([8, 5], 2048)])
def test_captured_and_replayed_with_other_lengths(gq, n, cap):
    """A captured call follows the lengths, queries and table in device memory."""
    import torch
    b = Batch(88, n, [cap - 7, cap // 2], 64, 2, 128)
    lens0 = b.lens.copy()
    q = queries(b, 8)
    cache, dq = b.cache(gq), to_dev(q)
    lens, q_start = b.dev()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        gq.gq_kv4_attn(cache, dq, lens, q_start, max_q=max(n))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = gq.gq_kv4_attn(cache, dq, lens, q_start, max_q=max(n))
    for step, new in enumerate(([cap - 7, cap // 2], [9, 1000], [700, 8], [cap, 65])):
        b.lens = np.array(new, np.int32)
        q = queries(b, 8)
        lens.copy_(to_dev(b.lens))
        dq.copy_(to_dev(q))
        g.replay()
        torch.cuda.synchronize()
        got = to_host(out).copy()
        keep, b.lens = b.lens, np.minimum(b.lens, b.table.shape[1] * 64).astype(np.int32)
        check_attention(b, got, q, 128 ** -0.5, True, 0)
        eager = to_host(gq.gq_kv4_attn(cache, dq, lens, q_start, max_q=max(n)))
        assert np.array_equal(got, eager), step
        b.lens = keep
    assert lens0[0] == cap - 7


def test_lengths_past_the_bound_are_taken_as_the_bound(gq):
    b = Batch(89, [1, 20], [100, 100], 16, 1, 64)
    q = queries(b, 2)
    want = to_host(run(gq, b, q, max_len=100))
    b.lens[:] = [2147483647, 101]
    got = to_host(run(gq, b, q, max_len=100))
    assert np.array_equal(got, want)
    b.lens[:] = [-5, -2147483648]
    assert not to_host(run(gq, b, q, max_len=100)).any()


def test_many_sequences(gq):
    n = 300
    lens = [1 + (i * 37) % 90 for i in range(n)]
    b = Batch(90, [1] * n, lens, 16, 1, 64, uniform=True)
    q = queries(b, 4)
    check_attention(b, to_host(run(gq, b, q, max_q=1)), q, 64 ** -0.5, True, 0)


def test_layer_as_it_is_used(gq):
    """A prompt and decode steps through append and attention together: what
    the cache holds is what attention reads, positions carried by both."""
    import torch
    import oracle.kv4 as o
    H, n_kv, hd, P = 8, 2, 64, 16
    rng = np.random.default_rng(91)
    freqs, m = gq.gq_rope_freqs(hd, 10000.0, gq.ROPE_YARN, 4.0, 64.0, 1.0, 32.0)
    rope = gq.Rope(freqs.cuda(), mscale=m)
    w = [(1 + 0.1 * rng.standard_normal(hd)).astype(np.float32) for _ in range(2)]
    b = Batch(92, [20, 37], [20, 37], P, n_kv, hd)
    b.table = rng.permutation(12).reshape(2, 6).astype(np.int32)
    b.pages = np.zeros((12, b.pages.shape[1]), np.uint8)
    cache = b.cache(gq)
    pages = b.pages.copy()
    for step, n in enumerate(([20, 37], [1, 1], [1, 1], [9, 4], [1, 0])):
        if step:
            b.lens = (b.lens + np.array(n)).astype(np.int32)
        b.q_start = np.concatenate(([0], np.cumsum(n))).astype(np.int32)
        b.n, b.n_tok = n, sum(n)
        x = rng.standard_normal((b.n_tok, H + 2 * n_kv, hd)).astype(np.float32)
        dev = to_dev(x)
        lens, q_start = b.dev()
        q = gq.gq_kv4_append(cache, dev[:, H:H + n_kv], dev[:, H + n_kv:], lens, q_start, rope=rope, k_norm=to_dev(w[1]),
                             q=dev[:, :H], q_norm=to_dev(w[0]), q_out=dev[:, :H])
        out = gq.gq_kv4_attn(cache, q, lens, q_start, max_q=max(n))
        where = o.rows(b.q_start, b.lens, b.n_tok)
        turned = o.rope(x[:, H:H + n_kv], [p for _, p in where], freqs.numpy(), False, m, w[1])
        for t, (s, p) in enumerate(where):
            for h in range(n_kv):
                o.store(pages, b.table[s, p // P], p % P, P, hd, h, 0, turned[t, h])
                o.store(pages, b.table[s, p // P], p % P, P, hd, h, 1, x[t, H + n_kv + h])
        assert np.array_equal(to_host(cache.pages).reshape(pages.shape), pages)
        check_attention(b, to_host(out), to_host(q), hd ** -0.5, True, 0, pages=pages)
    assert torch.cuda.is_available()


def test_refusals(gq):
    import torch
    b = Batch(93, [1, 2], [30, 40], 16, 2, 64)
    cache, q = b.cache(gq), to_dev(queries(b, 4))
    lens, q_start = b.dev()
    ok = dict(max_q=2)
    for bad in (dict(q=q.half()), dict(lens=lens.long()), dict(cache="x")):
        with pytest.raises(TypeError):
            gq.gq_kv4_attn(**(dict(cache=cache, q=q, lens=lens, q_start=q_start, **ok) | bad))
    for bad in (dict(q=q.cpu()), dict(q=q.transpose(0, 1)), dict(lens=lens[:1]), dict(q_start=q_start[:2]),
                dict(q_start=None), dict(q=q[..., :32].contiguous()), dict(out=q[:1]), dict(lens=lens.cpu())):
        with pytest.raises(ValueError):
            gq.gq_kv4_attn(**(dict(cache=cache, q=q, lens=lens, q_start=q_start, **ok) | bad))
    for bad in (dict(q=q[:, :3].contiguous()), dict(max_q=-1), dict(max_len=1 << 20), dict(window=-1),
                dict(out=q), dict(scale=float("nan"))):
        with pytest.raises(gq.GQError):
            gq.gq_kv4_attn(**(dict(cache=cache, q=q, lens=lens, q_start=q_start, **ok) | bad))
    with pytest.raises(gq.GQError):
        gq.KV4Cache(cache.pages, cache.table, 24, 2, 64)
    with pytest.raises(ValueError):
        gq.KV4Cache(cache.pages.view(-1)[:-16], cache.table, 16, 2, 64)
    assert gq.gq_kv4_attn(cache, q[:0], lens, torch.zeros_like(q_start), max_q=0).shape == (0, 4, 64)
