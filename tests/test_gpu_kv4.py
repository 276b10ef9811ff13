"""Rotary positions with per-head norms, appending to the 4-bit cache and
reading it back, against the 64-bit oracle on the GPU."""
import numpy as np
import pytest

import oracle.kv4 as o
from kv4_helpers import HALF, Batch, random_pages, to_dev, to_host

pytestmark = pytest.mark.gpu

FREQS = {r: (10000.0 ** (-np.arange(0, r, 2) / r)).astype(np.float32) for r in (0, 2, 8, 16, 20, 32, 40, 48, 64, 96, 128, 160, 192, 256)}


def rope_close(got, want, x_scale):
    """fp64 throughout and one rounding: half a step of the value, plus fp64's
    own noise against the head's magnitude (and fp32's smallest step)."""
    tol = HALF * np.abs(want) + 2.0 ** -44 * x_scale + 2.0 ** -149
    bad = np.abs(got.astype(np.float64) - want) > tol
    assert not bad.any(), (bad.sum(), np.abs(got - want)[bad].max())


@pytest.mark.parametrize("n,h,d,rot,inter,normed,first", [
    (1, 14, 64, 64, False, False, 777),
    (1, 1, 8, 8, True, True, 0),
    (3, 5, 24, 20, True, False, 11),
    (2, 9, 64, 32, False, True, 100000),
    (5, 3, 96, 96, False, True, 4095),
    (4, 2, 128, 0, False, True, 0),
    (7, 32, 128, 128, True, True, 1 << 20),
    (2, 3, 128, 40, False, False, -3),        # pairs that cross groups of eight channels
    (2, 3, 80, 20, False, True, 9),
    (1, 2, 160, 160, False, False, 5),
    (3, 17, 256, 192, False, True, 2_000_000_000),
    (2, 4, 256, 256, True, False, 131071),
    (1030, 3, 64, 64, False, True, 0),        # one workgroup per token
    (2, 3, 64, 2, True, False, 6),
])
def test_qk_rope(gq, n, h, d, rot, inter, normed, first):
    print(f"[kv4] rope n={n} h={h} d={d} rot={rot} inter={inter} norm={normed}", flush=True)
    rng = np.random.default_rng([1, n, h, d, rot])
    x = rng.standard_normal((n, h, d)).astype(np.float32) * np.float32(3.0)
    pos = (first + np.arange(n) * 3).astype(np.int32)
    w = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32) if normed else None
    rope = gq.Rope(to_dev(FREQS[rot]), interleaved=inter, mscale=1.25) if rot else None
    got = to_host(gq.gq_qk_rope(to_dev(x), to_dev(pos) if rot else None, rope, norm=None if w is None else to_dev(w),
                                eps=1e-5))
    want = o.rope(x, pos, FREQS[rot], inter, 1.25, w, 1e-5)
    rope_close(got, want, 1.25 * np.abs(want).max() * 2)


def test_qk_rope_in_place_and_strided(gq):
    # the q part of a fused q | k | v projection, turned where it lies
    import torch
    rng = np.random.default_rng(2)
    n, H, Hk, d = 6, 7, 2, 64
    x = rng.standard_normal((n, H + 2 * Hk, d)).astype(np.float32)
    pos = np.arange(n, dtype=np.int32) + 50
    dev = to_dev(x)
    q = dev[:, :H]
    rope = gq.Rope(to_dev(FREQS[64]))
    assert gq.gq_qk_rope(q, to_dev(pos), rope, out=q) is q
    got = to_host(dev)
    want = o.rope(x[:, :H], pos, FREQS[64])
    rope_close(got[:, :H], want, np.abs(x).max() * 2)
    assert np.array_equal(got[:, H:], x[:, H:])
    # the k part out of place into another stride
    big = torch.zeros((n, 5, d), device="cuda")
    gq.gq_qk_rope(to_dev(x)[:, H:H + Hk], to_dev(pos), rope, out=big[:, 1:3])
    got = to_host(big)
    rope_close(got[:, 1:3], o.rope(x[:, H:H + Hk], pos, FREQS[64]), np.abs(x).max() * 2)
    assert not got[:, 0].any() and not got[:, 3:].any()


def test_qk_rope_refuses(gq):
    import torch
    x = torch.zeros((2, 3, 64), device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    rope = gq.Rope(torch.ones(32, device="cuda"))
    for bad in (lambda: gq.gq_qk_rope(x.half(), pos, rope), lambda: gq.gq_qk_rope(x, pos.long(), rope),
                lambda: gq.gq_qk_rope(x, pos, torch.ones(32, device="cuda"))):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: gq.gq_qk_rope(x.cpu(), pos, rope), lambda: gq.gq_qk_rope(x.transpose(1, 2), pos, rope),
                lambda: gq.gq_qk_rope(x, pos[:1], rope), lambda: gq.gq_qk_rope(x[0], pos, rope),
                lambda: gq.gq_qk_rope(x, pos, rope, out=x[:1]), lambda: gq.gq_qk_rope(x, pos, rope, norm=x[0, 0, :8])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(gq.GQError):
        gq.gq_qk_rope(x[:, :, :24].contiguous(), pos, rope)       # rot past head_dim
    with pytest.raises(gq.GQError):
        gq.gq_qk_rope(x, None, rope)
    assert gq.gq_qk_rope(x[:0], pos, rope).shape == (0, 3, 64)


def _append(gq, batch, H, rot, inter, normed, seed, values=None, with_q=True, fused=True):
    """Appends rows to a copy of the batch's cache on the GPU and in the
    oracle: (pages got, pages wanted, q got, q wanted)."""
    rng = np.random.default_rng([77, seed])
    n, n_kv, hd, P = batch.n_tok, batch.n_kv, batch.hd, batch.P
    x = rng.standard_normal((n, H + 2 * n_kv, hd)).astype(np.float32) if values is None else values
    qw, kw = [(1 + 0.1 * rng.standard_normal(hd)).astype(np.float32) if normed else None for _ in range(2)]
    dev = to_dev(x)
    q, k, v = dev[:, :H], dev[:, H:H + n_kv], dev[:, H + n_kv:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    lens, q_start = batch.dev()
    cache = batch.cache(gq)
    rope = gq.Rope(to_dev(FREQS[rot]), interleaved=inter, mscale=1.125) if rot else None
    got_q = gq.gq_kv4_append(cache, k, v, lens, q_start, rope=rope, k_norm=None if kw is None else to_dev(kw),
                             q=q if with_q else None, q_norm=None if qw is None or not with_q else to_dev(qw), eps=1e-6)
    want = batch.pages.copy()
    where = o.rows(batch.q_start, batch.lens, n)
    pos = [0 if w is None else w[1] for w in where]
    kr = o.rope(x[:, H:H + n_kv], pos, FREQS[rot], inter, 1.125, kw)
    for t, w in enumerate(where):
        if w is None or w[1] < 0 or w[1] >= batch.table.shape[1] * P:
            continue
        page = int(batch.table[w[0], w[1] // P])
        if not 0 <= page < len(want):
            continue
        for h in range(n_kv):
            o.store(want, page, w[1] % P, P, hd, h, 0, kr[t, h])
            o.store(want, page, w[1] % P, P, hd, h, 1, x[t, H + n_kv + h])
    qr = o.rope(x[:, :H], pos, FREQS[rot], inter, 1.125, qw) if with_q else None
    return to_host(cache.pages).reshape(want.shape), want, None if got_q is None else to_host(got_q), qr, cache


@pytest.mark.parametrize("n,lens,P,H,n_kv,hd,rot,inter,normed", [
    ([1], [1], 16, 4, 1, 64, 64, False, False),
    ([1], [8192], 64, 32, 8, 128, 128, False, False),
    ([1, 1, 1], [16, 17, 333], 16, 14, 2, 64, 32, False, True),
    ([5, 0, 40], [5, 9, 50], 16, 3, 3, 96, 96, True, True),
    ([33, 17], [70, 17], 32, 2, 2, 256, 256, False, True),
    ([20], [20], 16, 1, 1, 32, 20, False, False),
    ([7], [1030], 1024, 2, 2, 160, 160, True, False),
    ([19], [19], 16, 5, 5, 224, 0, False, False),
])
def test_append_bytes(gq, n, lens, P, H, n_kv, hd, rot, inter, normed):
    # every byte of the pool, so nothing but the rows' slots changes
    print(f"[kv4] append n={n} lens={lens} P={P} kv={n_kv} hd={hd}", flush=True)
    b = Batch(len(n) + hd, n, lens, P, n_kv, hd)
    got, want, q, qr, cache = _append(gq, b, H, rot, inter, normed, hd)
    assert np.array_equal(got, want)
    rope_close(q, qr, 2.5 * np.abs(qr).max())
    # and read back: the held values, bit for bit
    K, V = gq.gq_kv4_read(cache, *b.dev()[:1], b.n_tok, b.dev()[1])
    K, V = to_host(K), to_host(V)
    for t, (s, p) in enumerate(o.rows(b.q_start, b.lens, b.n_tok)):
        page = int(b.table[s, p // P])
        for h in range(n_kv):
            assert np.array_equal(K[t, h], o.load(want, page, p % P, P, hd, h, 0))
            assert np.array_equal(V[t, h], o.load(want, page, p % P, P, hd, h, 1))


def test_append_keys_only_and_separate_tensors(gq):
    b = Batch(5, [3, 2], [30, 2], 16, 2, 64)
    got, want, q, _, _ = _append(gq, b, 0, 64, False, False, 5, with_q=False, fused=False)
    assert q is None and np.array_equal(got, want)


def test_append_many_tokens(gq):
    # over a thousand rows: one workgroup per token, all pages of a sequence
    b = Batch(6, [1100, 3], [1100, 8], 64, 1, 64)
    got, want, q, qr, _ = _append(gq, b, 2, 64, True, True, 6)
    assert np.array_equal(got, want)
    rope_close(q, qr, 2.5 * np.abs(qr).max())


def test_append_one_row_per_sequence(gq):
    # 70 sequences, no offsets; the same with offsets (searched 64 at a time)
    lens = [1 + (i * 13) % 60 for i in range(70)]
    for uniform in (True, False):
        b = Batch(7, [1] * 70, lens, 16, 1, 64, uniform=uniform)
        got, want, q, qr, _ = _append(gq, b, 1, 64, False, False, 7)
        assert np.array_equal(got, want)
        rope_close(q, qr, 2.5 * np.abs(qr).max())


def test_append_borders(gq):
    """Values where rounding decides: exact ties of the code and of the scale,
    equal magnitudes of both signs, zeros, subnormal scales, saturation,
    infinities and NaN. No rotation, so the inputs reach the blocks as they are."""
    rng = np.random.default_rng(8)
    hd, blocks = 64, []
    for d in (1.0, -0.5, 0.7109375, 2.0 ** -14, 2.0 ** -24, 3 * 2.0 ** -24, 255 * 2.0 ** -20):
        steps = np.concatenate((np.arange(-8, 8) + 0.5, np.arange(-8, 8)))
        x = rng.permutation(steps * d)
        x[np.abs(x) >= 8 * abs(d)] = 0.0
        x[int(rng.integers(32))] = -8 * d
        blocks.append(x)
    for m in (1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 2 - 2.0 ** -9, 1 + 2.0 ** -8 + 2.0 ** -20):
        blocks.append(rng.permutation(np.concatenate(([-8 * m], rng.uniform(-4, 4, 31)))))
    both = rng.uniform(-1, 1, 32)
    both[5], both[20] = 3.0, -3.0
    blocks += [both, -both, np.zeros(32), np.full(32, -0.0), rng.uniform(-1, 1, 32) * 1e-7, rng.uniform(-1, 1, 32) * 1e-44]
    blocks += [rng.uniform(-1, 1, 32) * 7e4, rng.uniform(-1, 1, 32) * 3e38, np.where(np.arange(32) == 7, np.inf, 1.0),
               np.where(np.arange(32) == 9, -np.inf, both), np.where(np.arange(32) == 11, np.nan, 1.0),
               np.where(np.arange(32) == 31, np.nan, np.inf)]
    if len(blocks) % 2:
        blocks.append(np.ones(32))
    n = len(blocks) // 2
    x = np.zeros((n, 2, hd), np.float32)
    x[:, 0] = np.array(blocks).reshape(n, hd).astype(np.float32)
    x[:, 1] = -x[:, 0]
    b = Batch(8, [n], [n], 16, 1, hd)
    with np.errstate(invalid="ignore"):
        got, want, _, _, _ = _append(gq, b, 0, 0, False, False, 8, values=x, with_q=False)
    # a NaN scale may have any payload: compare as values there
    diff = got != want
    code = 16 * hd // 2
    for p, i in zip(*np.nonzero(diff)):
        part, off = divmod(i, code + 16 * hd // 16)
        assert off >= code, "a code differs"
        lo = p, part * (code + 16 * hd // 16) + code + (off - code) // 2 * 2
        pair = [np.frombuffer(a[lo[0], lo[1]: lo[1] + 2].tobytes(), np.float16)[0] for a in (got, want)]
        assert np.isnan(pair).all() or (pair[0] == 0 and pair[1] == 0), pair


def test_append_and_read_bad_rows(gq):
    """Rows outside every sequence, positions outside the table, page numbers
    that are none: nothing is stored, other rows are unaffected."""
    import torch
    P, n_kv, hd, H = 16, 1, 64, 2
    b = Batch(9, [2, 3, 1, 2], [2, 20, 5, 33], P, n_kv, hd)
    b.table[1, 1] = len(b.pages)             # row 3 and 4 of sequence 1: positions 17..19
    b.table[2, 0] = -7
    b.lens[0] = 1                            # two rows, a cache of one: the first is at -1
    b.lens[3] = 2 + 16 * b.table.shape[1]    # one past the table, both rows
    x = np.random.default_rng(9).standard_normal((b.n_tok + 3, H + 2 * n_kv, hd)).astype(np.float32)
    dev = to_dev(x)
    lens, _ = b.dev()
    q_start = to_dev(b.q_start + 1)          # row 0 and the last two belong to none
    cache = b.cache(gq)
    q_out = torch.full((b.n_tok + 3, H, hd), 7.0, device="cuda")
    rope = gq.Rope(to_dev(FREQS[64]))
    gq.gq_kv4_append(cache, dev[:, H:H + 1], dev[:, H + 1:], lens, q_start, rope=rope, q=dev[:, :H], q_out=q_out)
    got, q = to_host(cache.pages).reshape(b.pages.shape), to_host(q_out)
    want = b.pages.copy()
    where = [None] + o.rows(b.q_start, b.lens, b.n_tok) + [None, None]
    turned = o.rope(x, [0 if w is None else w[1] for w in where], FREQS[64])
    K, V = torch.full((2, b.n_tok + 3, n_kv, hd), 9.0, device="cuda").unbind(0)
    for t, w in enumerate(where):
        if w is None or w[1] < 0 or w[1] >= b.table.shape[1] * P:
            assert (q[t] == 7.0).all(), t
            continue
        rope_close(q[t], turned[t, :H], 2.5 * np.abs(turned).max())
        page = int(b.table[w[0], w[1] // P])
        if 0 <= page < len(want):
            o.store(want, page, w[1] % P, P, hd, 0, 0, turned[t, H])
            o.store(want, page, w[1] % P, P, hd, 0, 1, x[t, H + 1])
    assert np.array_equal(got, want)
    gq.gq_kv4_read(cache, lens, b.n_tok + 3, q_start, K=K, V=V)
    K = to_host(K)
    for t, w in enumerate(where):
        if w is None or w[1] < 0 or w[1] >= b.table.shape[1] * P:
            assert (K[t] == 9.0).all(), t
        elif not 0 <= b.table[w[0], w[1] // P] < len(want):
            assert np.isnan(K[t]).all(), t
        else:
            assert np.array_equal(K[t, 0], o.load(want, b.table[w[0], w[1] // P], w[1] % P, P, hd, 0, 0))


def test_read_descending_offsets_and_whole_sequences(gq):
    import torch
    b = Batch(10, [40, 3, 100], [40, 3, 100], 32, 2, 96)
    cache = b.cache(gq)
    lens, q_start = b.dev()
    K, V = gq.gq_kv4_read(cache, lens, b.n_tok, q_start)
    for s in range(3):
        k, v = b.sequence(s)
        assert np.array_equal(to_host(K)[b.q_start[s]:b.q_start[s + 1]], k)
        assert np.array_equal(to_host(V)[b.q_start[s]:b.q_start[s + 1]], v)
    # offsets that descend, or leave the rows: those sequences have none
    for bad in ([0, 40, 30, 143], [-5, 40, 43, 143], [0, 40, 43, 999], [2147483647] * 4, [-2147483648] * 4):
        K = torch.full((b.n_tok, 2, 96), 9.0, device="cuda")
        V = K.clone()
        gq.gq_kv4_read(cache, lens, b.n_tok, to_dev(np.array(bad, np.int32)), K=K, V=V)
        torch.cuda.synchronize()
    only = to_host(gq.gq_kv4_read(cache, lens, b.n_tok, q_start, K=torch.empty_like(V))[0])
    assert np.array_equal(only[40:43], b.sequence(1)[0])


@pytest.mark.parametrize("n", [[40, 3], [1500, 2]])
def test_read_into_unaligned_outputs(gq, n):
    # four-byte aligned outputs, and only their rows are written
    import torch
    b = Batch(13, n, n, 64, 1, 64)
    lens, q_start = b.dev()
    size = b.n_tok * 64
    bufs = [torch.full((size + 2,), 9.0, device="cuda") for _ in range(2)]
    gq.gq_kv4_read(b.cache(gq), lens, b.n_tok, q_start, K=bufs[0][1:-1].view(-1, 1, 64), V=bufs[1][1:-1].view(-1, 1, 64))
    kv = [b.sequence(s) for s in range(2)]
    for i in range(2):
        got = to_host(bufs[i])
        assert got[0] == 9.0 and got[-1] == 9.0
        assert np.array_equal(got[1:-1].reshape(-1, 1, 64), np.concatenate((kv[0][i], kv[1][i])))


def test_append_captured(gq):
    """One decode step's append captured once and replayed with new tokens and
    lengths, eager work between; every replay's bytes against the oracle."""
    import torch
    b = Batch(11, [1, 1], [5, 30], 16, 2, 64, uniform=True)
    cache = b.cache(gq)
    lens, _ = b.dev()
    x = torch.zeros((2, 6, 64), device="cuda")
    rope = gq.Rope(to_dev(FREQS[64]))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        gq.gq_kv4_append(cache, x[:, 2:4], x[:, 4:], lens, rope=rope, q=x[:, :2])
    torch.cuda.synchronize()
    cache.pages.copy_(to_dev(b.pages))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q = gq.gq_kv4_append(cache, x[:, 2:4], x[:, 4:], lens, rope=rope, q=x[:, :2])
    want = b.pages.copy()
    rng = np.random.default_rng(11)
    for step in range(4):
        xs = rng.standard_normal((2, 6, 64)).astype(np.float32)
        x.copy_(to_dev(xs))
        b.lens[:] = [6 + step, 31 - 5 * step]
        lens.copy_(to_dev(b.lens))
        g.replay()
        torch.cuda.synchronize()
        turned = o.rope(xs, b.lens - 1, FREQS[64])
        for s_ in range(2):
            p = int(b.lens[s_]) - 1
            for h in range(2):
                o.store(want, b.table[s_, p // 16], p % 16, 16, 64, h, 0, turned[s_, 2 + h])
                o.store(want, b.table[s_, p // 16], p % 16, 16, 64, h, 1, xs[s_, 4 + h])
        assert np.array_equal(to_host(cache.pages).reshape(want.shape), want)
        rope_close(to_host(q), turned[:, :2], 2.5 * np.abs(turned).max())


def test_scales_of_another_writer(gq):
    """A cache with fp16 scales of 11 bits is read as it stands."""
    rng = np.random.default_rng(12)
    b = Batch(12, [50], [50], 16, 1, 64)
    code = 16 * 32
    pages = random_pages(rng, len(b.pages), 16, 1, 64).reshape(len(b.pages), 2, -1)
    pages[..., code:] = np.ascontiguousarray(rng.standard_normal((len(b.pages), 2, 32)).astype(np.float16)).view(np.uint8)
    b.pages = pages.reshape(len(b.pages), -1)
    K, _ = gq.gq_kv4_read(b.cache(gq), b.dev()[0], 50, b.dev()[1])
    assert np.array_equal(to_host(K), b.sequence(0)[0].astype(np.float32))
