"""The paged-cache calls where a first version went wrong: indices outside their
tables, rows that a mask hides, weights far below the largest, queries that are
not finite, padding.  Helpers and tolerances: test_paged.py."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle.kvq_oracle as O
from rotated_int4_kv_kvq_b200 import workloads as W
from test_paged import (BOTH, attend_f64, attend_tolerance, check_large, check_rounded,
                         gen, kvq, make_batch, make_pool, np64, poison, rows,
                         run_attend)  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore:invalid value:RuntimeWarning")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHAPES = [(64, 64), (64, 32), (128, 128), (128, 32), (256, 256), (256, 64)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,group", [(64, 64), (128, 32), (256, 128)])
def test_append_many_rows_far_positions(kvq, d, group, inter):
    """Positions far outside the table among many rows: those tokens are skipped
    whole and reported, the others come out as without them."""
    t, h, page = 2601, 4, 32
    signs = torch.from_numpy(W.make_signs(d)).cuda()
    x = rows(gen(6), t, h, d, torch.float16)
    slots = torch.arange(t, device="cuda")
    table = kvq.rope_table(3000, d // 2)
    pos = torch.arange(t, device="cuda", dtype=torch.int32)
    bad = [0, 31, 500, 1999, 2600]
    far = pos.clone()
    far[bad] = torch.tensor([2 ** 31 - 1, -2 ** 31, 3000, -1, 2 ** 30], device="cuda",
                            dtype=torch.int32)
    out = []
    for p, status in ((pos, 0), (far, 11)):
        cache = kvq.PagedCache.empty(t // page + 1, h, page, d, group, signs)
        for c in cache.tensors()[:4]:
            c.zero_()
        hat = torch.full_like(x, 9.0)
        kvq.kvq_paged_append(x, x, slots, cache, positions=p, cos_sin=table, interleaved=inter,
                             k_hat=hat)
        assert kvq.kvq_device_status() == status
        out.append([c.transpose(1, 2).flatten(0, 1)[:t] for c in cache.tensors()[:4]] + [hat])
    good = torch.ones(t, dtype=torch.bool, device="cuda")
    good[bad] = False
    for a, b in zip(*out):
        assert torch.equal(a[good], b[good])
    for b in out[1][:4]:
        assert (b[bad] == 0).all()
    assert (out[1][4][bad] == 9).all()


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("window", [0, 30])
def test_attend_hidden_values_of_any_size(kvq, dtype, d, group, window):
    """Values 2^30 (fp16: 2^18) times as large in rows that a token does not attend (later ones;
    with a window earlier ones too) leave its result as exact as any other."""
    n = 330
    cache = make_pool(kvq, d, 24, 2, 16, d, group, 0)
    table = make_batch(cache, 6, [n])
    at = torch.arange(n, device="cuda")
    page, off = table[0].long()[at // 16], at % 16
    a, b = (150, 260) if window else (100, n)
    cache.v_scales[page[a:b], :, off[a:b]] *= 2.0 ** (18 if dtype == torch.float16 else 30)
    cache.v_scales *= 2.0 ** -8  # what an fp16 result can hold
    q = rows(gen(3), n, 4, d, dtype) * 0.25
    dev = dict(device="cuda", dtype=torch.int32)
    got = kvq.kvq_paged_attend(q, cache, torch.tensor([0, n], **dev), torch.tensor([n], **dev),
                               table, max_q_len=n, window=window)
    assert kvq.kvq_device_status() == 0
    pools, tab = [x.cpu().numpy() for x in cache.tensors()[:4]], table.cpu().numpy()
    ref = O.attend_paged(np64(q), *pools, [0, n], [n], tab, cache.signs.cpu().numpy(), 0, group,
                         d ** -0.5, window)
    tol = attend_tolerance(np64(q), ref, pools, [0, n], [n], tab, cache, d ** -0.5, window, dtype)
    # A token that does attend some of them: besides 2^-11 of itself a weight times its
    # scale is off by half of fp16's smallest step, 2^-25, in units of 2^v, and 2^(v + 6)
    # is at most the largest attended scale S.  Each of up to n rows: 2^-31 S times a
    # code vector of at most 7 sqrt(d), over a sum of weights of at least 1.
    i = np.arange(n)
    none = (i < a) | (i - window >= b - 1) if window else i < a
    tol[~none] += n * 2.0 ** -31 * float(cache.v_scales.max()) * 7 * d ** 0.5
    assert none.sum() >= 100
    err = np.abs(np64(got) - ref)
    assert np.all(err <= tol), f"{(err / tol).max():.3g} x tolerance"


@pytest.mark.parametrize("kind", ["released", "unwritten"])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("nq,page,news,lens,window", [
    (4, 16, [1, 1], [1000, 333], 40), (2, 32, [4, 3], [700, 2000], 129), (1, 16, [1], [470], 1),
    (4, 16, [70, 33], [600, 433], 50), (3, 64, [300], [1500], 256), (16, 16, [9], [340], 17)])
def test_attend_pages_before_the_window(kvq, kind, d, group, nq, page, news, lens, window):
    """Pages that lie wholly before every token's window are not looked at: they may
    be released (-1), or hold whatever fresh memory does."""
    cache = make_pool(kvq, d + nq, sum(-(-m // page) for m in lens) + 2, 2, page, d, group, 0)
    table = make_batch(cache, 6, lens)
    poison(cache, table, lens)
    for s, (n, m) in enumerate(zip(news, lens)):
        free = max(0, m - n - window + 1) // page
        assert free > 0
        if kind == "released":
            table[s, :free] = -1
        else:
            gone = table[s, :free].long()
            cache.k_scales[gone], cache.v_scales[gone] = float("nan"), float("inf")
            cache.v_scales[gone[0]] = float("nan")
    cu = np.concatenate([[0], np.cumsum(news)]).tolist()
    q = rows(gen(nq), cu[-1], 2 * nq, d, torch.float16) * 0.25
    run_attend(kvq, cache, q, cu, lens, table, window=window)


@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("levels", [(16.5, 17.5), (20.0,), (14.0, 19.0)])
def test_attend_one_token_long_faint_tail(kvq, d, group, levels):
    """One early token outweighs each of the others by 2^14 to 2^20, all of them
    together weigh up to half as much as it."""
    n, seqs, heads, page = 16000, 48, 4, 64
    cache = make_pool(kvq, 8, n // page, heads, page, d, group, 0)
    # every key points the way of the first, every value but the first is the second's
    for t in (cache.k_packed, cache.k_scales, cache.v_packed, cache.v_scales):
        t[:, :, 2:] = t[:1, :, 1:2]
        t[1:, :, :2] = t[:1, :, 1:2]
    cache.k_packed[:] = cache.k_packed[:1, :, :1].clone()
    cache.k_scales[:] = cache.k_scales[:1, :, :1].clone()
    signs = cache.signs.cpu().numpy()
    key = O.dequant_rotated_f64(cache.k_packed[0, :, 0].cpu().numpy(),
                                cache.k_scales[0, :, 0].cpu().numpy(), signs, 0, group)
    top = 24.0  # score of the first token, the others 0 to 24 log 2 below
    q = torch.from_numpy(top * d ** 0.5 * key / (key ** 2).sum(-1, keepdims=True)).cuda().half()
    step = 1 - torch.tensor(levels, device="cuda", dtype=torch.float64) * np.log(2) / top
    f = step[torch.arange(n, device="cuda") % len(levels)].float().reshape(n // page, 1, page, 1)
    first = cache.k_scales[0, :, 0].clone()
    cache.k_scales.mul_(f)
    cache.k_scales[0, :, 0] = first
    table = torch.arange(n // page, device="cuda", dtype=torch.int32).repeat(seqs, 1)
    check_large(kvq, cache, q[None].repeat(seqs, 1, 1), list(range(seqs + 1)), [n] * seqs, table)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("rot", [O.SRFT, O.SRHT])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("max_q", [1, 1000])
def test_attend_queries_not_finite(kvq, dtype, rot, d, group, max_q):
    """A query with a NaN or an infinity gives NaN, whichever kernel takes it; its
    neighbours, and tokens that attend nothing, are what they were."""
    lens, nq = [900, 1, 0, 40], 4
    cache = make_pool(kvq, d, 70, 2, 16, d, group, rot)
    table = make_batch(cache, 9, lens)
    q = rows(gen(4), 4, 2 * nq, d, dtype) * 0.25
    args = (cache, torch.arange(5, device="cuda", dtype=torch.int32),
            torch.tensor(lens, device="cuda", dtype=torch.int32), table)
    want = kvq.kvq_paged_attend(q, *args, max_q_len=max_q)
    bad = [(0, 0, float("nan")), (0, 5, float("inf")), (1, 2, -float("inf")), (1, 7, float("inf")),
           (1, 4, float("nan")), (2, 3, float("nan")), (2, 1, float("inf"))]
    for t, h, x in bad:
        q[t, h, (7 * h + 3) % d] = x
        if t != 2:
            want[t, h] = float("nan")
    got = kvq.kvq_paged_attend(q, *args, max_q_len=max_q)
    assert kvq.kvq_device_status() == 0
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(), want.nan_to_num())
    assert (got[2] == 0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_norm_without_rotation_skips_padding(kvq, d):
    """Rows of tokens at negative positions stay, also where only a norm is asked for."""
    q, k = rows(gen(1), 6, 3, d, torch.float16), rows(gen(2), 6, 1, d, torch.float16)
    w = torch.randn(d, generator=gen(3), device="cuda")
    pos = torch.tensor([4, -1, 2 ** 31 - 1, 0, -7, -2 ** 31], device="cuda", dtype=torch.int32)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    kvq.kvq_qk_norm_rope(q, k, positions=pos, q_weight=w, k_weight=w, q_out=qo, k_out=ko)
    assert kvq.kvq_device_status() == 0  # without a table no position is outside it
    for x, o in ((q, qo), (k, ko)):
        assert (o[[1, 4, 5]] == 7.0).all()
        n = O.norm_rope(np64(x), np64(w), None, None)
        check_rounded(o[[0, 2, 3]], n[[0, 2, 3]], torch.float16,
                      np.abs(n).max(axis=-1, keepdims=True)[[0, 2, 3]])
    with pytest.raises(TypeError, match="int32"):
        kvq.kvq_qk_norm_rope(q, positions=pos.long(), q_weight=w)


@pytest.mark.parametrize("news", [[1, 1], [40, 30]])
def test_attend_window_past_32_bits(kvq, news):
    """A window of any size is a whole number of rows, not its low 32 bits."""
    cache = make_pool(kvq, 2, 20, 1, 16, 64, 64, 0)
    lens = [77, 150]
    table = make_batch(cache, 7, lens)
    q = rows(gen(3), sum(news), 2, 64, torch.float16) * 0.25
    args = (q, [0, news[0], sum(news)], lens, table)
    want = run_attend(kvq, cache, *args)
    for window in (2 ** 31, 2 ** 32 + 3, 2 ** 63 - 1, 2 ** 70):
        assert torch.equal(run_attend(kvq, cache, *args, window=window), want)
    assert torch.equal(run_attend(kvq, cache, *args, max_q=2 ** 40), want) or max(news) == 1
    for kw in (dict(window=-1), dict(window=-2 ** 32), dict(max_q=0), dict(max_q=-2 ** 32 + 1)):
        with pytest.raises(kvq.KVQError, match="BAD_SIZE"):
            run_attend(kvq, cache, *args, **kw)


def test_cache_fields_are_fixed(kvq):
    """The addresses that calls use are those of the tensors the cache shows."""
    signs = torch.from_numpy(W.make_signs(64)).cuda()
    cache = kvq.PagedCache.empty(4, 2, 16, 64, 32, signs)
    other = kvq.PagedCache.empty(9, 4, 32, 128, 128, torch.from_numpy(W.make_signs(128)).cuda(), 1)
    for name in ("k_packed", "v_scales", "signs", "rot", "n_pages", "group", "c", "ref", "other"):
        with pytest.raises(AttributeError, match="PagedCache"):
            setattr(cache, name, getattr(other, name, None))
    with pytest.raises(AttributeError, match="PagedCache"):
        del cache.k_packed
    cache.k_scales *= 2.0  # in place
    assert cache.k_packed.data_ptr() == cache.c.k_packed


FIRST = r'''
import sys
sys.path.insert(0, sys.argv[1])
import torch
from rotated_int4_kv_kvq_b200 import kvq, workloads as W
dev = torch.device("cuda", 0)
gen = torch.Generator(device=dev).manual_seed(5)
for d, g in ((64, 64), (128, 32), (256, 256)):
    signs = torch.from_numpy(W.make_signs(d)).to(dev)
    table = kvq.rope_table(9000, d)
    for new, heads in ((1, 1), (40, 2), (8000, 2)):
        pages = -(-new // 64)
        pt = torch.arange(pages, device=dev, dtype=torch.int32)[None]
        cu = torch.tensor([0, new], device=dev, dtype=torch.int32)
        ln = cu[1:].clone()
        x = torch.randn((new, 6 * heads, d), generator=gen, device=dev).half()
        q, k, v = x.split([4 * heads, heads, heads], 1)
        pos, slots = kvq.paged_rows(cu, ln, pt, 64, new)
        caches = []
        for _ in range(2):
            caches.append(kvq.PagedCache.empty(pages, heads, 64, d, g, signs))
            for t in caches[-1].tensors()[:4]:
                t.zero_()
        def layer(cache):
            kvq.kvq_paged_append(k, v, slots, cache, positions=pos, cos_sin=table)
            qr, _ = kvq.kvq_qk_norm_rope(q, positions=pos, cos_sin=table)
            return kvq.kvq_paged_attend(qr, cache, cu, ln, pt, max_q_len=new)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                o = layer(caches[0])
        torch.cuda.current_stream().wait_stream(side)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, layer(caches[1])), (d, g, new)
        for a, b in zip(caches[0].tensors(), caches[1].tensors()):
            assert torch.equal(a, b)
        del graph
assert kvq.kvq_device_status() == 0
print("ok")
'''


def test_first_calls_inside_graph_capture():
    """Whatever a call looks up once per process can be looked up during a capture."""
    r = subprocess.run([sys.executable, "-c", FIRST, ROOT], capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    assert r.stdout.strip().endswith("ok")
def test_key_output_without_keys(kvq):
    """What would come back unwritten is refused."""
    q, w = rows(gen(1), 3, 2, 64, torch.float16), torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="k_out"):
        kvq.kvq_qk_norm_rope(q, q_weight=w, k_out=torch.empty_like(q))


@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("news,lens,window", [([1, 1], [300, 77], 0), ([4, 3], [300, 77], 9),
                                              ([300, 20], [300, 77], 0), ([200, 60], [300, 77], 40)])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_attend_scales_not_finite(kvq, d, group, news, lens, window, which, value):
    """A cached row whose scale is not finite makes NaN of the tokens that attend it
    and leaves the others what they are."""
    cache = make_pool(kvq, d, 30, 2, 16, d, group, 0)
    table = make_batch(cache, 6, lens)
    # one row of each sequence (of one group of values in one KV head): the last but
    # one new token's, so that some tokens come before it and some after
    at = [m - (2 if n < 10 else n // 2) for n, m in zip(news, lens)]
    if news == [1, 1]:
        at = [100, 400]  # attended by the first; past the end of the second
    for s, t in enumerate(at):
        if t < lens[s]:
            scales = cache.k_scales if which == "k" else cache.v_scales
            scales[int(table[s, t // 16]), 0, t % 16, d // group - 1] = value
    q = rows(gen(4), sum(news), 4, d, torch.bfloat16) * 0.25
    cu = np.concatenate([[0], np.cumsum(news)]).tolist()
    with np.errstate(invalid="ignore"):
        got = run_attend(kvq, cache, q, cu, lens, table, window=window)
    for s, t in enumerate(at):
        p = np.arange(lens[s] - news[s], lens[s])
        bad = (p >= t) & ((p - t < window) if window else True) & (t < lens[s])
        mine = got[cu[s]:cu[s + 1]]
        assert mine[torch.from_numpy(bad), :2].isnan().all() and not mine[:, 2:].isnan().any()
        assert not mine[torch.from_numpy(~bad)].isnan().any()


@pytest.mark.parametrize("rot", [O.SRFT, O.SRHT])
@pytest.mark.parametrize("d,group", [(64, 64), (64, 32), (128, 128), (128, 64), (128, 32), (256, 256),
                                     (256, 128), (256, 64), (256, 32)])
@pytest.mark.parametrize("nq,news,lens,window", [(4, [300, 5], [1000, 700], 0), (1, [520], [900], 100)])
def test_attend_many_rows_fp16_keeps_its_bits(kvq, rot, d, group, nq, news, lens, window):
    """What a chunk's fp16 results are off by is their own rounding: uniform within half
    a step of at most 2^-10 |x|, so 2^-11 / sqrt(3) of the whole by the 2-norm, and 5%
    for all before it.  (Each row besides within its bound in the header.)"""
    cache = make_pool(kvq, d, sum(-(-m // 16) for m in lens), 4, 16, d, group, rot)
    table = make_batch(cache, 6, lens)
    cu = np.concatenate([[0], np.cumsum(news)]).tolist()
    q = (2 * torch.randn((cu[-1], 4 * nq, d), generator=gen(5), device="cuda")).half()
    dev = dict(device="cuda", dtype=torch.int32)
    got = kvq.kvq_paged_attend(q, cache, torch.tensor(cu, **dev), torch.tensor(lens, **dev), table,
                               max_q_len=max(news), window=window)
    assert kvq.kvq_device_status() == 0
    ref, mass, far = attend_f64(q, cache, cu, lens, table, window)
    err = (got.double() - ref).norm(dim=-1)
    tol = 2.0 ** -11 * ref.norm(dim=-1) + (torch.expm1(2 * 2.0 ** -15 * far) + 2.0 ** -15) * mass
    assert (err <= tol).all(), (err / tol).max().item()
    whole = (err.square().sum().sqrt() / ref.norm()).item()
    assert whole <= 1.05 * 2.0 ** -11 / 3 ** 0.5, whole


def test_paged_rows_captured(kvq):
    """Computed on the device alone: a captured call follows its inputs."""
    def batch(cu, lens, table):
        return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, lens, table)]
    first = batch([0, 3, 4], [20, 40], [[5, 9, 1], [3, 4, 2]])
    graph = torch.cuda.CUDAGraph()
    kvq.paged_rows(*first, 16, 6)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pos, slots = kvq.paged_rows(*first, 16, 6)
    for other in (first, batch([1, 1, 6], [0, 50], [[5, 9, 1], [-1, 4, 2]])):
        for a, b in zip(first, other):
            a.copy_(b)
        graph.replay()
        want = kvq.paged_rows(*(x.cpu() for x in other), 16, 6)
        assert pos.tolist() == want[0].tolist() and slots.tolist() == want[1].tolist()
    del graph
