"""The paged-cache calls without a GPU: argument checks on the host (fake
pointers below are never dereferenced), the binding's checks, and the host
helpers against plain loops."""

import ctypes

import numpy as np
import pytest
import torch

import oracle.kvq_oracle as O

A = 0x10000  # aligned fake device address (never dereferenced)


@pytest.fixture(scope="module")
def kvq():
    from rotated_int4_kv_kvq_b200 import build
    build.build()
    from rotated_int4_kv_kvq_b200 import kvq as mod
    return mod


def make_cache(kvq, **kw):
    f = dict(k_packed=A, v_packed=A, k_scales=A, v_scales=A, n_pages=8, n_kv_heads=2, page_size=16,
             d=64, group=32, signs=A, rot=0)
    f.update(kw)
    return kvq._PagedCacheC(*(f[n] for n, _ in kvq._PagedCacheC._fields_))


def make_rope(kvq, **kw):
    f = dict(cos_sin=A, n_pos=100, rot_dim=64, interleaved=0, eps=1e-6)
    f.update(kw)
    return kvq._RopeC(*(f[n] for n, _ in kvq._RopeC._fields_))


def norm_rope(kvq, rope="default", **kw):
    f = dict(q=A, k=A, dtype=0, n=4, hq=4, hk=2, d=64, qs=256, ks=128, pos=A, qw=A, kw=A, qo=A, ko=A,
             qos=256, kos=128)
    f.update(kw)
    r = make_rope(kvq) if rope == "default" else rope
    return kvq.lib.kvq_qk_norm_rope(f["q"], f["k"], f["dtype"], f["n"], f["hq"], f["hk"], f["d"],
                                    f["qs"], f["ks"], f["pos"], f["qw"], f["kw"],
                                    None if r is None else ctypes.byref(r), f["qo"], f["ko"],
                                    f["qos"], f["kos"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(d=96), 2), (dict(dtype=2), 12), (dict(dtype=-1), 12), (dict(n=-1), 7),
    (dict(n=1 << 31), 7), (dict(hq=0), 7), (dict(hk=-1), 7), (dict(hq=70000, qs=1 << 30), 7),
    (dict(qs=255), 7), (dict(qs=252), 7), (dict(qs=128), 7), (dict(kos=64), 7), (dict(qos=1 << 62), 7),
    (dict(n=1 << 30), 7),  # more rows than 2^31
    (dict(q=None), 1), (dict(k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(pos=None), 1),
    (dict(q=A + 8), 4), (dict(k=A + 2), 4), (dict(qo=A + 8), 4), (dict(qw=A + 4), 4), (dict(pos=A + 2), 4),
    (dict(n=0), 0), (dict(n=0, k=None, ko=None, hk=0), 0),
])
def test_norm_rope_host_checks(kvq, kw, expect):
    assert norm_rope(kvq, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(rot_dim=8), 7), (dict(rot_dim=24), 7), (dict(rot_dim=80), 7), (dict(n_pos=0), 7),
    (dict(eps=-1.0), 7), (dict(eps=float("nan")), 7), (dict(cos_sin=A + 8), 4),
])
def test_rope_host_checks(kvq, kw, expect):
    assert norm_rope(kvq, rope=make_rope(kvq, **kw)) == expect
    assert norm_rope(kvq, rope=None) == 1  # weights need the eps of a kvq_rope
    assert norm_rope(kvq, rope=None, qw=None, kw=None, pos=None, n=0) == 0


def append(kvq, cache=None, rope="default", **kw):
    f = dict(k=A, v=A, dtype=0, n=4, ks=128, vs=128, slots=A, pos=A, kw=A, kh=A, vh=A)
    f.update(kw)
    r = make_rope(kvq) if rope == "default" else rope
    c = make_cache(kvq) if cache is None else cache
    return kvq.lib.kvq_paged_append(f["k"], f["v"], f["dtype"], f["n"], f["ks"], f["vs"], f["slots"],
                                    f["pos"], f["kw"], None if r is None else ctypes.byref(r),
                                    ctypes.byref(c), f["kh"], f["vh"], None)


CACHE_CASES = [
    (dict(d=96), 2), (dict(group=16), 3), (dict(group=128), 3), (dict(rot=2), 5), (dict(n_pages=0), 7),
    (dict(n_pages=1 << 31), 7), (dict(n_kv_heads=0), 7), (dict(page_size=8), 7), (dict(page_size=24), 7),
    (dict(page_size=512), 7), (dict(k_packed=None), 1), (dict(v_scales=None), 1), (dict(signs=None), 1),
    (dict(k_packed=A + 8), 4), (dict(v_packed=A + 4), 4), (dict(k_scales=A + 4), 4),
]


@pytest.mark.parametrize("kw,expect", CACHE_CASES)
def test_cache_host_checks(kvq, kw, expect):
    c = make_cache(kvq, **kw)
    assert append(kvq, cache=c) == expect
    assert attend(kvq, cache=c) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=3), 12), (dict(n=-1), 7), (dict(n=1 << 31), 7), (dict(ks=64), 7), (dict(vs=132), 7),
    (dict(k=None), 1), (dict(v=None), 1), (dict(slots=None), 1), (dict(pos=None), 1),
    (dict(k=A + 8), 4), (dict(slots=A + 4), 4), (dict(kw=A + 4), 4), (dict(vh=A + 2), 4),
    (dict(n=0), 0), (dict(n=0, kh=None, vh=None, kw=None), 0),
])
def test_append_host_checks(kvq, kw, expect):
    assert append(kvq, **kw) == expect


def test_append_without_rope(kvq):
    assert append(kvq, rope=None) == 1  # a weight needs the eps of a kvq_rope
    assert append(kvq, rope=None, kw=None, pos=None, n=0) == 0


def attend(kvq, cache=None, **kw):
    f = dict(q=A, dtype=0, n=4, qs=256, cu=A, kl=A, pt=A, ns=2, mp=4, nq=2, mq=4, win=0, sc=0.125, o=A,
             os=256, ws=A, wb=1 << 40)
    f.update(kw)
    c = make_cache(kvq) if cache is None else cache
    return kvq.lib.kvq_paged_attend(f["q"], f["dtype"], f["n"], f["qs"], ctypes.byref(c), f["cu"],
                                    f["kl"], f["pt"], f["ns"], f["mp"], f["nq"], f["mq"], f["win"],
                                    f["sc"], f["o"], f["os"], f["ws"], f["wb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=2), 12), (dict(n=-1), 7), (dict(nq=0), 7), (dict(nq=65, qs=1 << 14, os=1 << 14), 7),
    (dict(qs=128), 7), (dict(os=252), 7), (dict(ns=-1), 7), (dict(ns=1 << 17), 7), (dict(mp=-1), 7),
    (dict(mp=1 << 28), 7), (dict(mq=0), 7), (dict(win=-1), 7), (dict(sc=float("nan")), 7),
    (dict(sc=float("inf")), 7), (dict(q=None), 1), (dict(o=None), 1), (dict(cu=None), 1),
    (dict(kl=None), 1), (dict(pt=None), 1), (dict(q=A + 2), 4), (dict(o=A + 8), 4), (dict(cu=A + 2), 4),
    (dict(ws=A + 16), 4), (dict(n=0), 0), (dict(ns=0), 0),
])
def test_attend_host_checks(kvq, kw, expect):
    assert attend(kvq, **kw) == expect


def test_workspace_query_checks(kvq):
    ws = kvq.lib.kvq_paged_attend_workspace
    assert ws(4, 2, 2, 96, 1) == -2
    assert ws(-1, 2, 2, 64, 1) == -7
    assert ws(4, 2, 65, 64, 1) == -7
    assert ws(4, 2, 2, 64, 0) == -7


def test_binding_checks_before_launch(kvq):
    x = torch.zeros((2, 4, 64), dtype=torch.float16)
    with pytest.raises(TypeError, match="CUDA tensor"):
        kvq.kvq_qk_norm_rope(x)
    with pytest.raises(ValueError, match="k_packed"):
        kvq.PagedCache(None, None, None, None, None)
    with pytest.raises(TypeError, match="CUDA tensor"):
        kvq.PagedCache.empty(2, 1, 16, 64, 32, torch.ones(64, dtype=torch.int8))


def test_refused_stream_leaves_the_device(kvq, monkeypatch):
    """A call that fails on its stream argument does not change the current device."""
    entered = []

    class Guard:
        def __init__(self, dev):
            pass

        def __enter__(self):
            entered.append(1)

        def __exit__(self, *_):
            entered.pop()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    with pytest.raises((TypeError, ValueError)):
        kvq._enter(1, "no stream")
    assert not entered
    raw, guard = kvq._enter(1, 1234)
    assert raw == 1234 and isinstance(guard, Guard) and entered == [1]
    assert kvq._enter(0, 1234) == (1234, None)


@pytest.mark.parametrize("group", [48, 40, 0, -32, 96, 100, 256])
def test_cache_of_no_such_group(kvq, group):
    """A group that does not divide d is refused, not replaced by one that does."""
    with pytest.raises(ValueError, match="group"):
        kvq.PagedCache.empty(4, 2, 16, 128, group, torch.ones(128, dtype=torch.int8))


def test_rope_table(kvq):
    t = kvq.rope_table(5000, 32, 500000.0, device="cpu").numpy()
    for p in (0, 1, 777, 4999):
        a = p * 500000.0 ** (-np.arange(16) / 16)
        # one rounding to fp32 of values of size at most 1, and a 64-bit angle
        assert np.abs(t[p, :16] - np.cos(a)).max() <= 2.0 ** -25 + 1e-11
        assert np.abs(t[p, 16:] - np.sin(a)).max() <= 2.0 ** -25 + 1e-11


def test_paged_rows(kvq):
    cu = torch.tensor([0, 3, 3, 7], dtype=torch.int32)
    ln = torch.tensor([20, 5, 4], dtype=torch.int32)
    pt = torch.tensor([[4, 2, 9], [1, 0, 0], [7, 0, 0]], dtype=torch.int32)
    pos, slots = kvq.paged_rows(cu, ln, pt, 16, 9)  # tokens 7 and 8 belong to nobody
    assert pos.tolist() == [17, 18, 19, 0, 1, 2, 3, -1, -1] and pos.dtype == torch.int32
    assert slots.tolist() == [33, 34, 35, 112, 113, 114, 115, -1, -1] and slots.dtype == torch.int64


NOWHERE = 1 << 62  # past every pool: the append skips and reports it


def test_paged_rows_past_the_table(kvq):
    """A token whose page the table does not have must not land on another's row."""
    i32 = dict(dtype=torch.int32)
    # two pages of 16: positions 32 and 33 have none
    pos, slots = kvq.paged_rows(torch.tensor([0, 3, 4], **i32), torch.tensor([34, 40], **i32),
                                torch.tensor([[5, 9], [3, 4]], **i32), 16, 5)
    assert pos.tolist() == [31, 32, 33, 39, -1]
    assert slots.tolist() == [9 * 16 + 15, NOWHERE, NOWHERE, NOWHERE, -1]
    # a page that was never given, or was released
    pos, slots = kvq.paged_rows(torch.tensor([0, 3], **i32), torch.tensor([17], **i32),
                                torch.tensor([[2, -1]], **i32), 16, 3)
    assert pos.tolist() == [14, 15, 16] and slots.tolist() == [46, 47, NOWHERE]
    # more new tokens than rows: those before position 0 have none
    pos, slots = kvq.paged_rows(torch.tensor([0, 3], **i32), torch.tensor([2], **i32),
                                torch.tensor([[2]], **i32), 16, 3)
    assert pos.tolist()[1:] == [0, 1] and pos[0] < 0 and slots.tolist() == [-1, 32, 33]


def test_paged_rows_of_nothing(kvq):
    """A padded batch without sequences, a table without pages, no tokens."""
    i32 = dict(dtype=torch.int32)
    pos, slots = kvq.paged_rows(torch.zeros(1, **i32), torch.zeros(0, **i32),
                                torch.zeros((0, 4), **i32), 16, 3)
    assert pos.tolist() == [-1] * 3 and pos.dtype == torch.int32
    assert slots.tolist() == [-1] * 3 and slots.dtype == torch.int64
    pos, slots = kvq.paged_rows(torch.tensor([0, 1], **i32), torch.tensor([1], **i32),
                                torch.zeros((1, 0), **i32), 16, 2)
    assert pos.tolist() == [0, -1] and slots.tolist() == [NOWHERE, -1]
    pos, slots = kvq.paged_rows(torch.tensor([0, 0], **i32), torch.tensor([7], **i32),
                                torch.zeros((1, 2), **i32), 16, 0)
    assert pos.shape == slots.shape == (0,)


def test_paged_rows_offsets_out_of_order(kvq):
    """Only a sequence that holds a token says where it goes."""
    i32 = dict(dtype=torch.int32)
    for cu in ([0, 6, 2, 8], [3, 1, 8, 8], [0, 9, 4, 2], [-4, 2, 4, 6]):
        lens, table = [20, 20, 20], [[1, 2], [3, 4], [5, 6]]
        pos, slots = kvq.paged_rows(torch.tensor(cu, **i32), torch.tensor(lens, **i32),
                                    torch.tensor(table, **i32), 16, 8)
        for t, (p, s) in enumerate(zip(pos.tolist(), slots.tolist())):
            may = {(-1, -1)}
            for b, e, n, row in zip(cu, cu[1:], lens, table):
                if b <= t < e:
                    q = n - e + t
                    may.add((q, row[q // 16] * 16 + q % 16) if q >= 0 else (q, -1))
            assert (p, s) in may


def test_oracle_norm_rope_turns_pairs():
    """A rotation keeps each pair's length and adds angles: position p on top
    of position p' is p + p'."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 64))
    i = np.arange(16) / 16
    ang = np.arange(50)[:, None] * 100.0 ** -i
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    for inter in (False, True):
        one = O.norm_rope(x, None, [3, 10, 20], table, inter)
        two = O.norm_rope(one, None, [5, 0, 29], table, inter)
        ref = O.norm_rope(x, None, [8, 10, 49], table, inter)
        assert np.abs(two - ref).max() < 1e-12
        assert np.array_equal(one[..., 32:], x[..., 32:])
    w = rng.standard_normal(64)
    n = O.norm_rope(x, w, None, None, eps=0.0)
    assert np.abs(((n / w) ** 2).mean(-1) - 1).max() < 1e-12


def test_oracle_attend_paged_is_attend_decode_for_one_token():
    rng = np.random.default_rng(1)
    d, g, page = 64, 32, 16
    signs = np.where(rng.random(d) < 0.5, -1, 1).astype(np.int8)
    pool = [rng.integers(0, 256, (6, 2, page, d // 2), dtype=np.uint8),
            rng.random((6, 2, page, d // g)).astype(np.float32)] * 2
    q = rng.standard_normal((1, 4, d)).astype(np.float16)
    table = np.array([[3, 0, 5]], dtype=np.int32)
    got = O.attend_paged(q, *pool, [0, 1], [37], table, signs, 0, g, 0.2)
    flat = [x[table[0]].transpose(1, 0, 2, 3).reshape(2, 48, -1) for x in pool]
    ref = O.attend_decode(q.reshape(2, 2, d), *flat, 37, signs, 0, g, 0.2)
    err = np.abs(got.reshape(2, 2, d) - ref.astype(np.float64))
    assert np.all(err <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -25)  # ref is rounded to fp16
