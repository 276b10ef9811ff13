"""The entry points of the rotary positions and the 4-bit cache reject bad
arguments on the host (fake pointers: a call that passes every check would
launch, so none here does), and the host-only functions' values. CPU only."""
import ctypes
import math

import numpy as np
import pytest

import gguf_block_quant_gq_amd as gq

A = [0x1000000 * (i + 1) for i in range(16)]   # far apart, 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return gq.load_library()


def rejected(status):
    assert status != gq.GQ_ERR_DEVICE, "the call passed every host check"
    return status


def rope(freqs=A[9], rot=64, interleaved=0, mscale=1.0):
    return gq._RopeStruct(freqs, rot, interleaved, mscale)


def kv4(pages=A[0], n_pages=8, page_tokens=16, n_kv=2, head_dim=64, table=A[1], table_stride=4, n_seq=2):
    return gq._KV4Struct(pages, n_pages, page_tokens, n_kv, head_dim, table, table_stride, n_seq)


def qk(lib, x=A[2], xs=128, n=4, h=2, d=64, pos=A[3], r=0, w=None, eps=1e-6, out=A[4], os=128):
    r = rope() if r == 0 else r
    return rejected(lib.gq_qk_rope(x, xs, n, h, d, pos, ctypes.addressof(r) if r else None, w, eps, out, os, None))


def append(lib, c=0, k=A[2], ks=128, v=A[3], vs=128, n=4, start=A[5], lens=A[6], r=None, kw=None, q=None, qs=128, h=0,
           qw=None, qo=None, qos=128, eps=1e-6):
    c = kv4() if c == 0 else c
    return rejected(lib.gq_kv4_append(ctypes.addressof(c) if c else None, k, ks, v, vs, n, start, lens,
                                      ctypes.addressof(r) if r else None, kw, q, qs, h, qw, qo, qos, eps, None))


def read(lib, c=0, n=4, start=A[5], lens=A[6], K=A[2], V=A[3]):
    c = kv4() if c == 0 else c
    return rejected(lib.gq_kv4_read(ctypes.addressof(c) if c else None, n, start, lens, K, V, None))


def attn(lib, c=0, q=A[2], qs=256, h=4, n=4, start=A[5], lens=A[6], max_q=4, max_len=64, scale=0.125, causal=1,
         window=0, out=A[3], os=256, ws=A[4], wsb=1 << 30):
    c = kv4() if c == 0 else c
    return rejected(lib.gq_kv4_attn(ctypes.addressof(c) if c else None, q, qs, h, n, start, lens, max_q, max_len,
                                    scale, causal, window, out, os, ws, wsb, None))


def test_page_bytes(lib):
    assert gq.gq_kv4_page_bytes(16, 2, 64) == 16 * 2 * 72
    assert gq.gq_kv4_page_bytes(64, 8, 128) == 64 * 8 * 144
    for bad in ((8, 2, 64), (24, 2, 64), (2048, 2, 64), (0, 2, 64), (-16, 2, 64), (16, 0, 64), (16, -1, 64),
                (16, 65536, 64), (16, 2, 0), (16, 2, 48), (16, 2, 288), (16, 2, -64)):
        assert gq.gq_kv4_page_bytes(*bad) < 0, bad


def test_qk_rope_arguments(lib):
    S, N, AL, OV = gq.GQ_ERR_SHAPE, gq.GQ_ERR_NULL, gq.GQ_ERR_ALIGN, gq.GQ_ERR_OVERLAP
    for bad in (dict(n=-1), dict(n=(1 << 30) + 1), dict(h=-1), dict(h=1 << 30), dict(d=4), dict(d=60), dict(d=264),
                dict(d=0), dict(xs=127), dict(os=64), dict(xs=1 << 62), dict(w=A[7], eps=-1.0),
                dict(w=A[7], eps=math.nan), dict(r=rope(rot=66)), dict(r=rope(rot=63)), dict(r=rope(rot=-2)),
                dict(r=rope(interleaved=2))):
        assert qk(lib, **bad) == S, bad
    for bad in (dict(x=None), dict(out=None), dict(pos=None), dict(r=rope(freqs=None))):
        assert qk(lib, **bad) == N, bad
    for bad in (dict(x=A[2] + 2), dict(out=A[4] + 1), dict(pos=A[3] + 2), dict(w=A[7] + 1), dict(r=rope(freqs=A[9] + 2))):
        assert qk(lib, **bad) == AL, bad
    for bad in (dict(out=A[2] + 4), dict(out=A[2], os=256), dict(out=A[3]), dict(out=A[9]), dict(w=A[4] + 8),
                dict(x=A[4] + 512 * 3 + 256)):
        assert qk(lib, **bad) == OV, bad
    for none in (dict(n=0, x=None), dict(h=0, x=None, out=None)):
        assert qk(lib, **none) == gq.GQ_OK
    # the q and k parts of one buffer's rows, 192 floats apart: the parts are
    # disjoint, their ends are not; one float more and they touch
    assert qk(lib, x=A[2], xs=192, out=A[2] + 4 * 64, os=192) == OV


def test_append_arguments(lib):
    S, N, AL, OV = gq.GQ_ERR_SHAPE, gq.GQ_ERR_NULL, gq.GQ_ERR_ALIGN, gq.GQ_ERR_OVERLAP
    for bad in (kv4(n_pages=-1), kv4(n_pages=0), kv4(n_pages=1 << 31), kv4(page_tokens=20), kv4(head_dim=80), kv4(n_kv=0),
                kv4(table_stride=-1), kv4(table_stride=(1 << 26) + 1), kv4(n_seq=-1)):
        for call in (append, read, attn):
            assert call(lib, c=bad) == S
    for call in (append, read, attn):
        assert call(lib, c=None) == N
        assert call(lib, n=-1) == S
        assert call(lib, n=3, start=None) == S                 # one row per sequence
        assert call(lib, lens=None) == N
        assert call(lib, c=kv4(pages=None)) == N
        assert call(lib, c=kv4(table=None)) == N
        assert call(lib, c=kv4(pages=A[0] + 8)) == AL
        assert call(lib, c=kv4(table=A[1] + 2)) == AL
        assert call(lib, lens=A[6] + 1) == AL
        assert call(lib, start=A[5] + 2) == AL
        assert call(lib, n=0) == gq.GQ_OK
        assert call(lib, c=kv4(n_seq=0)) == gq.GQ_OK
    for bad in (dict(ks=127), dict(vs=1), dict(kw=A[7], eps=-1.0), dict(r=rope(rot=66)), dict(q=A[7], h=-1, qo=A[8]),
                dict(q=A[7], h=4, qo=A[8]), dict(q=A[7], h=1 << 29, qo=A[8], qs=1 << 40, qos=1 << 40)):
        assert append(lib, **bad) == S, bad
    for bad in (dict(k=None), dict(v=None), dict(q=A[7], h=2), dict(r=rope(freqs=None))):
        assert append(lib, **bad) == N, bad
    for bad in (dict(k=A[2] + 2), dict(v=A[3] + 1), dict(kw=A[7] + 1), dict(q=A[7] + 2, h=2, qo=A[8]),
                dict(q=A[7], h=2, qo=A[8] + 3)):
        assert append(lib, **bad) == AL, bad
    q = dict(q=A[7], h=2, qs=128)
    for bad in (dict(k=A[0] + 64), dict(v=A[0] + 8 * 2304 - 4), dict(lens=A[0]), dict(start=A[0] + 16), dict(kw=A[0]),
                dict(**q, qo=A[7] + 4), dict(**q, qo=A[7], qos=256), dict(**q, qo=A[2]), dict(**q, qo=A[3] + 64),
                dict(**q, qo=A[6]), dict(**q, qo=A[5]), dict(**q, qo=A[1]), dict(**q, qo=A[0]),
                dict(**q, qo=A[8], kw=A[8] + 4), dict(**q, qo=A[8], qw=A[8] + 4), dict(q=A[0], h=2, qo=A[8])):
        assert append(lib, **bad) == OV, bad
    # rows of one buffer, 320 floats apart, in place: q at 0, k at 128, v one float short of its place
    f = A[10]
    assert append(lib, q=f, qs=320, h=2, qo=f, qos=320, k=f + 4 * 127, ks=320, v=f + 4 * 256, vs=320) == OV


def test_read_arguments(lib):
    assert read(lib, K=None, V=None) == gq.GQ_OK
    assert read(lib, K=A[2] + 2) == gq.GQ_ERR_ALIGN
    assert read(lib, V=A[2] + 4 * 4 * 128 - 4) == gq.GQ_ERR_OVERLAP
    for o in (A[0], A[1], A[5], A[6]):
        assert read(lib, K=o) == gq.GQ_ERR_OVERLAP
        assert read(lib, V=o) == gq.GQ_ERR_OVERLAP


def test_attention_arguments(lib):
    S, N, AL, OV = gq.GQ_ERR_SHAPE, gq.GQ_ERR_NULL, gq.GQ_ERR_ALIGN, gq.GQ_ERR_OVERLAP
    for bad in (dict(h=0), dict(h=3), dict(h=-2), dict(max_q=-1), dict(max_len=-1), dict(max_len=65), dict(window=-1),
                dict(scale=math.nan), dict(scale=math.inf), dict(qs=255), dict(os=255), dict(wsb=-1),
                dict(max_q=1 << 30)):
        assert attn(lib, **bad) == S, bad
    for bad in (dict(q=None), dict(out=None)):
        assert attn(lib, **bad) == N, bad
    for bad in (dict(q=A[2] + 2), dict(out=A[3] + 2)):
        assert attn(lib, **bad) == AL, bad
    for bad in (dict(out=A[2]), dict(out=A[2] + 256), dict(out=A[0]), dict(out=A[1]), dict(out=A[5]), dict(out=A[6])):
        assert attn(lib, **bad) == OV, bad
    assert attn(lib, max_q=0) == gq.GQ_OK


def test_attention_workspace(lib):
    # a long context of one sequence is split; its workspace is asked for
    c = kv4(table_stride=1024, n_seq=1)
    need = lib.gq_kv4_attn_ws_bytes(ctypes.addressof(c), 4, 1, 16384)
    assert need > 0
    args = dict(c=c, start=None, n=1, max_q=1, max_len=16384)
    assert attn(lib, **args, wsb=need - 1) == gq.GQ_ERR_SHAPE
    assert attn(lib, **args, ws=None) == gq.GQ_ERR_NULL
    assert attn(lib, **args, ws=A[4] + 8) == gq.GQ_ERR_ALIGN
    for o in (A[0], A[1], A[2], A[3], A[6]):
        assert attn(lib, **args, ws=o) == gq.GQ_ERR_OVERLAP
    for bad in (dict(h=3), dict(max_q=-1), dict(max_len=16385)):
        a = dict(h=4, max_q=1, max_len=16384) | bad
        assert lib.gq_kv4_attn_ws_bytes(ctypes.addressof(c), a["h"], a["max_q"], a["max_len"]) < 0
    assert lib.gq_kv4_attn_ws_bytes(None, 4, 1, 16) < 0


def test_python_binding_refuses_cpu_tensors():
    import torch
    with pytest.raises((ValueError, RuntimeError)):
        gq.KV4Cache(torch.zeros(2304, dtype=torch.uint8), torch.zeros((1, 1), dtype=torch.int32), 16, 2, 64)
    with pytest.raises((ValueError, RuntimeError)):
        gq.Rope(torch.zeros(8))


# ------------------------------------------------------------------- freqs
def test_freqs_plain_and_linear():
    f, m = gq.gq_rope_freqs(128, 10000.0)
    want = 10000.0 ** (-np.arange(0, 128, 2) / 128)
    # correctly rounded but for pow's own last bit
    assert np.abs(f.numpy() / want - 1).max() <= 2.0 ** -24 + 1e-15 and m == 1.0
    g, m = gq.gq_rope_freqs(128, 10000.0, gq.ROPE_LINEAR, 4.0)
    assert np.array_equal(g.numpy(), f.numpy() / 4) and m == 1.0
    assert gq.gq_rope_freqs(0)[0].numel() == 0


def test_freqs_bands():
    rot, base, factor, ctx, lo, hi = 128, 500000.0, 8.0, 8192.0, 1.0, 4.0
    f = gq.gq_rope_freqs(rot, base, gq.ROPE_BANDS, factor, ctx, lo, hi)[0].numpy().astype(float)
    for p in range(rot // 2):
        plain = base ** (-2 * p / rot)
        wave = 2 * math.pi / plain
        if wave < ctx / hi:
            want = plain
        elif wave > ctx / lo:
            want = plain / factor
        else:
            s = (ctx / wave - lo) / (hi - lo)
            want = (1 - s) * plain / factor + s * plain
        assert abs(f[p] / want - 1) <= 2.0 ** -23, p
    assert f[0] == 1.0 and abs(f[-1] * factor / base ** (-126 / 128) - 1) < 1e-6


def test_freqs_yarn():
    rot, base, factor, ctx, lo, hi = 64, 10000.0, 16.0, 4096.0, 1.0, 32.0
    f, m = gq.gq_rope_freqs(rot, base, gq.ROPE_YARN, factor, ctx, lo, hi)
    f = f.numpy().astype(float)
    plain = base ** (-np.arange(0, rot, 2) / rot)
    assert m == pytest.approx(0.1 * math.log(16.0) + 1, abs=1e-7)
    turns = ctx * plain / (2 * math.pi)
    # pairs of clearly more than hi turns are kept, of clearly fewer than lo interpolated,
    # and the share kept falls linearly over the pair index between
    first = math.floor(rot * math.log(ctx / (hi * 2 * math.pi)) / (2 * math.log(base)))
    last = math.ceil(rot * math.log(ctx / (lo * 2 * math.pi)) / (2 * math.log(base)))
    assert turns[first] >= hi and turns[last] <= lo
    share = (f / plain - 1 / factor) / (1 - 1 / factor)
    p = np.arange(rot // 2)
    assert np.abs(share - np.clip(1 - (p - first) / (last - first), 0, 1)).max() < 1e-6


def test_freqs_arguments(lib):
    buf = (ctypes.c_float * 64)()
    m = ctypes.c_float()

    def call(rot=64, base=1e4, scaling=gq.ROPE_YARN, factor=4.0, ctx=4096.0, lo=1.0, hi=32.0, out=ctypes.addressof(buf)):
        return lib.gq_rope_freqs(rot, base, scaling, factor, ctx, lo, hi, out, ctypes.addressof(m))

    assert call() == gq.GQ_OK
    for bad in (dict(rot=-2), dict(rot=3), dict(rot=1 << 21), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
                dict(scaling=-1), dict(scaling=4), dict(factor=0.5), dict(factor=math.nan), dict(ctx=0.0),
                dict(lo=0.0), dict(hi=1.0), dict(hi=math.inf), dict(ctx=math.nan)):
        assert call(**bad) == gq.GQ_ERR_SHAPE, bad
    assert call(out=None) == gq.GQ_ERR_NULL
    assert call(scaling=gq.ROPE_PLAIN, factor=math.nan, ctx=0.0, lo=0.0) == gq.GQ_OK   # not read
    with pytest.raises(gq.GQError):
        gq.gq_rope_freqs(7)
