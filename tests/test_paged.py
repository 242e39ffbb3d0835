"""The paged-cache calls on a B200 against the float64 oracle: norm and position
rotation, append, attention of new tokens, and the three in a row.

Tolerances.  A result rounded once to a type with unit roundoff u
(torch.finfo(t).eps / 2) is off by u |x|; fp32 arithmetic before it adds
F32 = 2e-6 of the largest value that enters (sums of at most 256 terms, a few
operations each).  Attention adds, for scores formed from queries rounded to
11 bits, |ds_t| <= 2^-11 sm_scale sum_i |Rq_i y_K,t,i| =: D, so that a weight
is off by a factor within exp(+-2 D) after normalization, and 2^-10 for
weights rounded to 11 bits (each one's own, and its share in the sum); both
weigh sum_t p_t |y_V,t|, taken through |R^T| <= 1 per value as its 2-norm.
"""

import numpy as np
import pytest
import torch

import oracle.kvq_oracle as O
from parity import TIE_WINDOW, SCALE_RTOL
from rotated_int4_kv_kvq_b200 import workloads as W

pytestmark = [pytest.mark.gpu,
              # rows past a sequence's end hold NaN and infinity, the oracle's pools too
              pytest.mark.filterwarnings("ignore:invalid value:RuntimeWarning")]

F32 = 2e-6
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half the smallest step
BOTH = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def kvq():
    from rotated_int4_kv_kvq_b200 import kvq as mod
    return mod


def np64(t):
    return t.double().cpu().numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(g, tokens, heads, d, dtype):
    x = torch.randn((tokens, heads, d), generator=g, device="cuda")
    x[..., 3] *= 20  # an outlier channel
    return x.to(dtype)


def check_rounded(got, ref, dtype, scale):
    err = np.abs(np64(got) - ref)
    tol = UNIT[dtype] * np.abs(ref) + TINY[dtype] + F32 * scale
    assert np.all(err <= tol), f"{(err / tol).max():.3g} x tolerance"


# ------------------------------------------------------------ norm and rope ---

@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("d,rot_dim,inter,qn,kn", [
    (64, 64, False, False, False), (64, 32, True, True, True), (128, 128, False, True, True),
    (128, 64, False, True, False), (128, 16, True, False, True), (256, 256, False, True, True),
    (256, 48, False, False, True), (256, 112, True, True, True), (256, 0, False, True, True)])
@pytest.mark.parametrize("tokens,hq,hk", [(1, 1, 0), (1, 4, 1), (5, 12, 2), (333, 33, 3)])
def test_norm_rope(kvq, dtype, d, rot_dim, inter, qn, kn, tokens, hq, hk):
    g = gen(d + rot_dim + tokens + hq)
    qkv = rows(g, tokens, hq + 2 * hk, d, dtype)  # a fused projection
    q, k = qkv[:, :hq], (qkv[:, hq:hq + hk] if hk else None)
    table = kvq.rope_table(4000, rot_dim) if rot_dim else None
    pos = torch.randint(0, 4000, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    qw = torch.randn(d, generator=g, device="cuda") if qn else None
    kw = torch.randn(d, generator=g, device="cuda") if kn else None
    before = qkv.clone()
    qo, ko = kvq.kvq_qk_norm_rope(q, k, positions=pos, cos_sin=table, interleaved=inter,
                                  q_weight=qw, k_weight=kw, eps=1e-5)
    torch.cuda.synchronize()
    assert kvq.kvq_device_status() == 0 and torch.equal(qkv, before)
    tab = None if table is None else table.cpu().numpy()
    for x, w, out in ((q, qw, qo), (k, kw, ko)):
        if x is None:
            assert out is None
            continue
        ref = O.norm_rope(np64(x), None if w is None else np64(w), pos.cpu().numpy(), tab, inter, 1e-5)
        n = O.norm_rope(np64(x), None if w is None else np64(w), None, None, False, 1e-5)
        check_rounded(out, ref, dtype, np.abs(n).max(axis=-1, keepdims=True))
    # in place, inside the projection
    kvq.kvq_qk_norm_rope(q, k, positions=pos, cos_sin=table, interleaved=inter, q_weight=qw,
                         k_weight=kw, eps=1e-5, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(q, qo) and (k is None or torch.equal(k, ko))
    assert torch.equal(qkv[:, hq + hk:], before[:, hq + hk:])  # the values beside them


def test_norm_rope_skips_padding_and_bad_positions(kvq):
    q = rows(gen(1), 6, 3, 128, torch.float16)
    table = kvq.rope_table(50, 128)
    pos = torch.tensor([4, -1, 49, 50, -7, 2 ** 31 - 1], device="cuda", dtype=torch.int32)
    out = torch.full_like(q, 7.0)
    kvq.kvq_qk_norm_rope(q, positions=pos, cos_sin=table, q_out=out)
    assert kvq.kvq_device_status() == 11 and kvq.kvq_device_status() == 0
    for t in (1, 3, 4, 5):
        assert (out[t] == 7.0).all()
    ref = O.norm_rope(np64(q[[0, 2]]), None, [4, 49], table.cpu().numpy())
    check_rounded(out[[0, 2]], ref, torch.float16, np.abs(ref).max(axis=-1, keepdims=True))
    pos[3:] = -1
    kvq.kvq_qk_norm_rope(q, positions=pos, cos_sin=table, q_out=out)
    assert kvq.kvq_device_status() == 0  # padding is no error


def test_norm_rope_zero_row_and_no_tokens(kvq):
    q = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    out, none = kvq.kvq_qk_norm_rope(q, q_weight=w)
    assert none is None and (out == 0).all()
    assert kvq.kvq_qk_norm_rope(q[:0], q_weight=w)[0].shape == (0, 1, 64)


# ------------------------------------------------------------------- append ---

def check_append(kvq, cache, slots, values, hats, dtype):
    """values: K and V [T, H, d] in float64 as the forward step takes them."""
    d, g, signs = cache.d, cache.group, cache.signs.cpu().numpy()
    s = slots.cpu().numpy()
    pg, off = s // cache.page_size, s % cache.page_size
    for (packed, scales), x, hat in zip(((cache.k_packed, cache.k_scales),
                                         (cache.v_packed, cache.v_scales)), values, hats):
        p = packed.cpu().numpy()[pg, :, off].reshape(-1, d // 2)
        sc = scales.cpu().numpy()[pg, :, off].reshape(-1, d // g)
        y = O.rotate(O.sign_flip(x.reshape(-1, d), signs), cache.rot)
        q_ref, s_ref = O.quantize_groups(y, g)
        # the key's norm and rotation in fp32 come before the transform's own rounding
        assert np.all(np.abs(sc - s_ref) <= 4 * SCALE_RTOL * s_ref)
        q = O.unpack_nibbles(p)
        bad = q != q_ref
        if bad.any():
            assert np.abs(q[bad].astype(int) - q_ref[bad]).max() == 1
            assert O.near_tie_distance(y, s_ref, g)[bad].max() < TIE_WINDOW
            assert bad.mean() < 1e-4 or bad.sum() <= 2
        if hat is not None:
            ref = O.dequant_rotated_f64(p, sc, signs, cache.rot, g).reshape(x.shape)
            check_rounded(hat, ref, dtype, np.abs(x).max(axis=-1, keepdims=True))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("rot", [O.SRFT, O.SRHT])
@pytest.mark.parametrize("d,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128),
                                     (256, 32), (256, 64), (256, 128), (256, 256)])
@pytest.mark.parametrize("tokens,heads,page,norm,rot_dim,inter",
                         [(1, 1, 16, True, 64, False), (37, 3, 32, False, 0, False),
                          (50, 2, 256, True, 32, True), (200, 5, 64, False, 48, False),
                          # enough rows for a thread a row; a last, partial tile
                          (2601, 4, 64, True, 64, False), (5159, 2, 16, False, 32, True)])
def test_append(kvq, dtype, rot, d, group, tokens, heads, page, norm, rot_dim, inter):
    g = gen(d + group + tokens)
    signs = torch.from_numpy(W.make_signs(d)).cuda()
    pages = tokens // page + 3
    cache = kvq.PagedCache.empty(pages, heads, page, d, group, signs, rot)
    for t in (cache.k_packed, cache.v_packed):
        t.fill_(0x5A)
    for t in (cache.k_scales, cache.v_scales):
        t.fill_(float("nan"))
    qkv = rows(g, tokens, 3 * heads, d, dtype)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens]
    table = kvq.rope_table(5000, rot_dim) if rot_dim else None
    pos = torch.randint(0, 5000, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randn(d, generator=g, device="cuda") if norm else None
    kh, vh = torch.empty((tokens, heads, d), dtype=dtype, device="cuda"), None
    if tokens != 37:
        vh = torch.empty_like(kh)
    kvq.kvq_paged_append(k, v, slots, cache, positions=pos, cos_sin=table, interleaved=inter,
                         k_weight=w, k_hat=kh, v_hat=vh)
    torch.cuda.synchronize()
    assert kvq.kvq_device_status() == 0
    k64 = O.norm_rope(np64(k), None if w is None else np64(w), pos.cpu().numpy(),
                      None if table is None else table.cpu().numpy(), inter)
    check_append(kvq, cache, slots, (k64, np64(v)), (kh, vh), dtype)
    keep = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    keep[slots] = False
    for t in (cache.k_packed, cache.v_packed):
        assert (t.transpose(1, 2).flatten(0, 1)[keep] == 0x5A).all()
    for t in (cache.k_scales, cache.v_scales):
        assert t.transpose(1, 2).flatten(0, 1)[keep].isnan().all()


@pytest.mark.parametrize("d,group", [(64, 64), (128, 32), (256, 128)])
def test_append_many_rows_skips_the_same(kvq, d, group):
    """Padding, bad slots and bad positions among many rows: the rows written,
    and their codes up to ties, are those of calls of few rows."""
    t, h, page = 2601, 4, 32
    signs = torch.from_numpy(W.make_signs(d)).cuda()
    x = rows(gen(6), t, h, d, torch.float16)
    slots = torch.randperm(t + 50, generator=gen(7), device="cuda")[:t]
    slots[5], slots[40], slots[41], slots[2600] = -1, 10 ** 6, -(2 ** 40), 1 << 40
    table = kvq.rope_table(3000, d // 2)
    pos = torch.arange(t, device="cuda", dtype=torch.int32)
    pos[77], pos[78] = 3000, -3
    out = []
    for parts in ([(0, t)], [(a, min(a + 100, t)) for a in range(0, t, 100)]):
        cache = kvq.PagedCache.empty(t // page + 3, h, page, d, group, signs)
        for c in cache.tensors()[:4]:
            c.zero_()
        hat = torch.full_like(x, 9.0)
        for a, b in parts:
            kvq.kvq_paged_append(x[a:b], x[a:b], slots[a:b], cache, positions=pos[a:b],
                                 cos_sin=table, k_hat=hat[a:b])
        assert kvq.kvq_device_status() == 11
        out.append((cache, hat))
    (c0, h0), (c1, h1) = out
    skipped = [5, 40, 41, 77, 78, 2600]
    assert (h0[skipped] == 9).all() and (h1[skipped] == 9).all()
    assert torch.equal(h0 == 9, h1 == 9) or ((h0 == 9) != (h1 == 9)).float().mean() < 1e-3
    for a, b in zip(c0.tensors()[:4], c1.tensors()[:4]):
        if a.dtype == torch.uint8:
            assert (a != b).float().mean() < 1e-3
        else:
            assert torch.equal(a > 0, b > 0) and ((a - b).abs() <= 4e-6 * b).all()
    assert int((c0.v_scales > 0).any(-1).sum()) == (t - len(skipped)) * h


def test_append_is_the_forward_step(kvq):
    """Without norm and rotation a page row has the codes of kvq_rot_quant_fwd
    (up to ties) and kvq_dequant_rot_inv reads the pool back as k_hat."""
    d, group = 128, 32
    signs = torch.from_numpy(W.make_signs(d)).cuda()
    cache = kvq.PagedCache.empty(4, 2, 16, d, group, signs)
    x = rows(gen(5), 64, 2, d, torch.float16)
    kh, vh = torch.empty_like(x), torch.empty_like(x)
    slots = torch.arange(64, device="cuda")
    kvq.kvq_paged_append(x, x, slots, cache, k_hat=kh, v_hat=vh)
    packed, scales = kvq.kvq_rot_quant_fwd(x.reshape(-1, d), signs, 0, group)
    mine = cache.k_packed.transpose(1, 2).reshape(-1, d // 2)
    assert torch.equal(cache.k_packed, cache.v_packed) and torch.equal(kh, vh)
    assert (mine != packed).float().mean() < 1e-3
    s = cache.k_scales.transpose(1, 2).reshape(-1, d // group)
    assert ((s - scales).abs() <= 1e-6 * scales).all()
    back = kvq.kvq_dequant_rot_inv(cache.k_packed.reshape(-1, d // 2),
                                   cache.k_scales.reshape(-1, d // group), signs, 0, group)
    back = back.reshape(4, 2, 16, d).transpose(1, 2).reshape(64, 2, d)
    big = x.double().abs().amax(-1, keepdim=True)
    assert ((back.double() - kh.double()).abs() <= 2 * (2.0 ** -11 + F32) * big).all()


def test_append_skips_padding_and_bad_slots(kvq):
    d = 64
    signs = torch.from_numpy(W.make_signs(d)).cuda()
    cache = kvq.PagedCache.empty(2, 1, 16, d, 32, signs)
    for t in cache.tensors()[:4]:
        t.zero_()
    x = rows(gen(2), 5, 1, d, torch.bfloat16)
    kh = torch.full_like(x, 3.0)
    slots = torch.tensor([7, -1, 32, 2 ** 40, 31], device="cuda")
    kvq.kvq_paged_append(x, x, slots, cache, k_hat=kh)
    assert kvq.kvq_device_status() == 11
    assert (kh[1:4] == 3.0).all() and (kh[0] != 3.0).any() and (kh[4] != 3.0).any()
    written = (cache.k_scales.flatten(0, 2) > 0).any(-1)
    assert written.nonzero().flatten().tolist() == [7, 31]
    # a position outside the table: the token is skipped whole, its value too
    for t in cache.tensors()[:4]:
        t.zero_()
    table = kvq.rope_table(10, 64)
    pos = torch.tensor([3, 10, 2, -1, 9], device="cuda", dtype=torch.int32)
    kvq.kvq_paged_append(x, x, torch.arange(5, device="cuda"), cache, positions=pos, cos_sin=table)
    assert kvq.kvq_device_status() == 11
    for s in (cache.k_scales, cache.v_scales):
        assert (s.flatten(0, 2) > 0).any(-1).nonzero().flatten().tolist() == [0, 2, 4]


def test_append_far_in_a_large_pool(kvq):
    """Rows whose byte offsets pass 32 bits."""
    d, page = 256, 256
    signs = torch.from_numpy(W.make_signs(d)).cuda()
    pages = (1 << 32) // (page * d // 2) + 40
    cache = kvq.PagedCache.empty(pages, 1, page, d, 256, signs)
    x = rows(gen(3), 4, 1, d, torch.float16)
    n = pages * page
    slots = torch.tensor([n - 1, n - 300, 5, n // 2], device="cuda")
    kh, vh = torch.empty_like(x), torch.empty_like(x)
    kvq.kvq_paged_append(x, x, slots, cache, k_hat=kh, v_hat=vh)
    assert kvq.kvq_device_status() == 0
    at, off = slots // page, slots % page
    small = kvq.PagedCache(cache.k_packed[at, :, off][:, :, None].repeat(1, 1, 16, 1),
                           cache.k_scales[at, :, off][:, :, None].repeat(1, 1, 16, 1),
                           cache.v_packed[at, :, off][:, :, None].repeat(1, 1, 16, 1),
                           cache.v_scales[at, :, off][:, :, None].repeat(1, 1, 16, 1), signs)
    check_append(kvq, small, torch.arange(4, device="cuda") * 16, (np64(x), np64(x)), (kh, vh),
                 torch.float16)
    # and attention finds them there
    q = rows(gen(4), 1, 1, d, torch.float16)
    table = torch.tensor([[pages - 1]], device="cuda", dtype=torch.int32)
    cache.k_packed[-1].zero_(), cache.v_packed[-1].zero_()
    cache.k_scales[-1].zero_(), cache.v_scales[-1].zero_()
    kvq.kvq_paged_append(x[:1], x[:1], slots[:1], cache)
    run_attend(kvq, cache, q, [0, 1], [256], table)


# ---------------------------------------------------------------- attention ---

def attend_tolerance(q, ref, pools, cu, lens, table, cache, scale, window, dtype):
    """See the module's text; per (token, head)."""
    signs, g, nq = cache.signs.cpu().numpy(), cache.group, q.shape[1] // cache.n_kv_heads
    yk = [O.dequantize_groups(O.unpack_nibbles(pools[0][p].reshape(-1, cache.d // 2)),
                              pools[1][p].reshape(-1, pools[1].shape[-1]), g)
          .reshape(cache.n_kv_heads, cache.page_size, cache.d) for p in range(len(pools[0]))]
    yv = [np.linalg.norm(O.dequantize_groups(
        O.unpack_nibbles(pools[2][p].reshape(-1, cache.d // 2)),
        pools[3][p].reshape(-1, pools[3].shape[-1]), g), axis=-1)
        .reshape(cache.n_kv_heads, cache.page_size) for p in range(len(pools[0]))]
    rq = O.rotate(O.sign_flip(q, signs), cache.rot)
    tol = np.zeros(q.shape[:2])
    for s in range(len(lens)):
        n = cu[s + 1] - cu[s]
        t = np.arange(lens[s])
        pg = np.asarray(table[s])[t // cache.page_size]
        good = (pg >= 0) & (pg < len(pools[0]))
        pg, off = np.where(good, pg, 0), t % cache.page_size
        k = np.stack([yk[p][:, o] for p, o in zip(pg, off)], 1) if lens[s] else None
        v = np.stack([yv[p][:, o] for p, o in zip(pg, off)], 1) if lens[s] else None
        for i in range(cu[s], cu[s + 1]):
            p = lens[s] - n + i - cu[s]
            see = good & (t <= p) & ((t > p - window) if window else True)
            if not see.any():
                continue
            for h in range(q.shape[1]):
                kk, vv = k[h // nq][see], v[h // nq][see]
                w = scale * kk @ rq[i, h]
                w = np.exp(w - w.max())
                w /= w.sum()
                D = 2.0 ** -11 * abs(scale) * (np.abs(kk) @ np.abs(rq[i, h])).max()
                tol[i, h] = (np.expm1(2 * D) + 2.0 ** -10 + F32) * (w @ vv)
    return tol[..., None] + UNIT[dtype] * np.abs(ref) + TINY[dtype]


def run_attend(kvq, cache, q, cu, lens, table, scale=None, window=0, max_q=None, out=None, **kw):
    dtype, d = q.dtype, cache.d
    sc = d ** -0.5 if scale is None else scale
    dev = dict(device="cuda", dtype=torch.int32)
    cu_t, len_t = torch.tensor(cu, **dev), torch.tensor(lens, **dev)
    n = max([1] + [b - a for a, b in zip(cu, cu[1:])]) if max_q is None else max_q
    got = kvq.kvq_paged_attend(q, cache, cu_t, len_t, table, max_q_len=n, window=window,
                               sm_scale=scale, out=out, **kw)
    torch.cuda.synchronize()
    assert kvq.kvq_device_status() == 0
    used = sorted({int(p) for r, m in zip(table.tolist(), lens)
                   for p in r[:-(-m // cache.page_size)] if 0 <= p < cache.n_pages})
    small = np.full(cache.n_pages + 1, -1)
    small[used] = np.arange(len(used))
    pools = [x[used].cpu().numpy() if used else x[:1].cpu().numpy() for x in cache.tensors()[:4]]
    tab = table.cpu().numpy().astype(np.int64)
    tab = small[np.where((tab < 0) | (tab >= cache.n_pages), cache.n_pages, tab)]
    ref = O.attend_paged(np64(q), *pools, cu, lens, tab, cache.signs.cpu().numpy(), cache.rot,
                         cache.group, sc, window)
    own = ~np.isnan(ref[:, 0, 0])
    tol = attend_tolerance(np64(q), np.nan_to_num(ref), pools, cu, lens, tab, cache, sc, window, dtype)
    err = np.abs(np64(got) - ref)[own]
    assert np.all(err <= tol[own]), f"{np.nanmax(err / tol[own]):.3g} x tolerance"
    return got


def make_pool(kvq, seed, pages, heads, page, d, group, rot):
    """A pool with a model's keys and values in every page."""
    g = gen(seed)
    signs = torch.from_numpy(W.make_signs(d)).cuda()
    cache = kvq.PagedCache.empty(pages, heads, page, d, group, signs, rot)
    n = pages * page
    x = torch.randn((n, 2 * heads, d), generator=g, device="cuda")
    x[..., 3] *= 10
    x = x.half()
    kvq.kvq_paged_append(x[:, :heads], x[:, heads:], torch.arange(n, device="cuda"), cache)
    return cache


def make_batch(cache, seed, lens):
    """A page table over a shuffled pool; entries past a sequence's pages are
    out of range and must not be read."""
    need = [-(-m // cache.page_size) for m in lens]
    order = torch.randperm(cache.n_pages, generator=gen(seed), device="cuda").tolist()
    assert sum(need) <= cache.n_pages
    table = torch.full((len(lens), max(need + [1])), 1 << 30, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = torch.tensor(order[at:at + n])
        at += n
    return table.cuda()


def poison(cache, table, lens):
    """Rows past each sequence's end, and pages of no sequence, hold the worst
    that fresh memory can: NaN and infinite scales."""
    used = torch.zeros((cache.n_pages, cache.page_size), dtype=torch.bool)
    for r, m in zip(table.tolist(), lens):
        for t in range(m):
            used[r[t // cache.page_size], t % cache.page_size] = True
    free = ~used.cuda()
    for t, bad in ((cache.k_scales, float("nan")), (cache.v_scales, float("inf"))):
        t.masked_fill_(free[:, None, :, None], bad)


SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128),
          (256, 256)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("rot", [O.SRFT, O.SRHT])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("nq,heads,page,lens", [
    (1, 1, 16, [1]), (4, 2, 32, [37, 1, 300]), (6, 1, 64, [1000]), (8, 2, 16, [129, 128, 127, 16])])
def test_attend_one_token(kvq, dtype, rot, d, group, nq, heads, page, lens):
    cache = make_pool(kvq, d + nq, sum(-(-m // page) for m in lens) + 2, heads, page, d, group, rot)
    table = make_batch(cache, 5, lens)
    poison(cache, table, lens)
    q = rows(gen(nq), len(lens), heads * nq, d, dtype) * 0.25
    run_attend(kvq, cache, q, list(range(len(lens) + 1)), lens, table)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("rot", [O.SRFT, O.SRHT])
@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("nq,heads,page,news,lens,window", [
    (1, 2, 16, [5, 1, 3], [5, 40, 130], 0),          # drafted tokens, one from position 0
    (2, 1, 32, [130, 0, 7], [130, 9, 300], 0),       # a whole prompt, an idle sequence, a chunk
    (4, 1, 64, [70, 33], [333, 33], 50),             # a sliding window
    (3, 2, 16, [100], [257], 1),                     # each token sees itself alone
    (16, 1, 16, [9], [140], 0)])
def test_attend_chunk(kvq, dtype, rot, d, group, nq, heads, page, news, lens, window):
    cache = make_pool(kvq, d + nq, sum(-(-m // page) for m in lens) + 2, heads, page, d, group, rot)
    table = make_batch(cache, 6, lens)
    poison(cache, table, lens)
    cu = np.concatenate([[0], np.cumsum(news)]).tolist()
    q = rows(gen(nq), cu[-1], heads * nq, d, dtype) * 0.25
    run_attend(kvq, cache, q, cu, lens, table, window=window)


@pytest.mark.parametrize("news", [[9, 1], [40, 200]])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30, 5000])
def test_attend_wide_window(kvq, news, window):
    """A window wider than everything is none, for tokens before position 0 too."""
    lens = [7, 250]
    cache = make_pool(kvq, 2, 20, 1, 16, 64, 64, 0)
    table = make_batch(cache, 7, lens)
    q = rows(gen(3), sum(news), 2, 64, torch.float16) * 0.25
    a = run_attend(kvq, cache, q, [0, news[0], sum(news)], lens, table, window=window)
    b = run_attend(kvq, cache, q, [0, news[0], sum(news)], lens, table)
    assert torch.equal(a, b)


@pytest.mark.parametrize("d,group", [(64, 64), (128, 32), (256, 256)])
@pytest.mark.parametrize("max_q", [1, 2, 16, 1000])
def test_attend_any_hint(kvq, d, group, max_q):
    """max_q_len chooses a kernel and nothing else."""
    lens, news = [500, 7, 64], [40, 1, 64]
    cache = make_pool(kvq, 1, 50, 2, 16, d, group, 0)
    table = make_batch(cache, 7, lens)
    q = rows(gen(2), sum(news), 6, d, torch.float16) * 0.25
    run_attend(kvq, cache, q, [0, 40, 41, 105], lens, table, max_q=max_q)


@pytest.mark.parametrize("news", [[1, 1], [40, 30]])
@pytest.mark.parametrize("scale,ramp", [(0.0, 0.0), (2.0, 0.0), (-0.3, 0.0), (0.5, 4.0)])
def test_attend_flat_sharp_and_rising(kvq, news, scale, ramp):
    """No preference, nearly one-hot weights, a negative scale, and scores that
    rise along the sequence so that the running maximum moves."""
    d, lens = 128, [700, 444]
    cache = make_pool(kvq, 3, 24, 2, 64, d, 128, 0)
    table = make_batch(cache, 8, lens)
    if ramp:
        for r, m in zip(table.tolist(), lens):
            for i, p in enumerate(r[:-(-m // 64)]):
                cache.k_scales[p] *= 1 + ramp * i
    q = rows(gen(9), sum(news), 4, d, torch.float16) * 0.1
    run_attend(kvq, cache, q, [0, news[0], sum(news)], lens, table, scale=scale)


@pytest.mark.parametrize("news", [[1, 1, 1], [30, 2, 20]])
@pytest.mark.parametrize("d,group", [(64, 32), (128, 128), (256, 64)])
def test_attend_scales_of_all_sizes(kvq, news, d, group):
    """Values whose scales differ by many orders of magnitude between rows,
    zero rows, and a row that outweighs all others."""
    lens = [400, 150, 300]
    cache = make_pool(kvq, 4, 60, 1, 16, d, group, 0)
    g = gen(10)
    e = torch.randint(-12, 5, cache.v_scales.shape[:3], generator=g, device="cuda")
    cache.v_scales *= torch.exp2(e.float())[..., None]
    cache.v_scales *= 1000.0
    cache.k_scales[torch.rand(cache.k_scales.shape[:3], generator=g, device="cuda") < 0.2] = 0.0
    table = make_batch(cache, 11, lens)
    cu = np.concatenate([[0], np.cumsum(news)]).tolist()
    q = rows(gen(12), cu[-1], 2, d, torch.bfloat16) * 0.25
    run_attend(kvq, cache, q, cu, lens, table)


def test_attend_strides_and_rows_of_nobody(kvq):
    """Queries inside a fused projection, an output inside a wider buffer, and
    tokens before the first and behind the last sequence, left as they were."""
    d, lens = 64, [50, 20]
    cache = make_pool(kvq, 5, 8, 2, 16, d, 64, 0)
    table = make_batch(cache, 13, lens)
    for cu in ([2, 3, 5], [1, 30, 50]):
        lens = [max(lens[0], cu[1] - cu[0]), max(lens[1], cu[2] - cu[1])]
        wide = rows(gen(14), 60, 4 + 4, d, torch.float16) * 0.25
        buf = torch.full((60, 6, d), 9.0, dtype=torch.float16, device="cuda")
        run_attend(kvq, cache, wide[:, :4], cu, lens, table, out=buf[:, 1:5])
        assert (buf[:cu[0]] == 9).all() and (buf[cu[-1]:] == 9).all()
        assert (buf[:, 0] == 9).all() and (buf[:, 5] == 9).all()


@pytest.mark.parametrize("news", [[1, 1], [20, 20]])
def test_attend_empty_and_bad(kvq, news):
    """Tokens that attend nothing get zeros; bad pages, lengths and offsets are
    reported and not followed."""
    d = 128
    cache = make_pool(kvq, 6, 8, 1, 16, d, 128, 0)
    dev = dict(device="cuda", dtype=torch.int32)
    table = torch.tensor([[0, 1, 2], [3, 4, 5]], **dev)
    n = sum(news)
    q = rows(gen(15), n, 2, d, torch.float16) * 0.25
    cu = torch.tensor([0, news[0], n], **dev)

    def call(cu=cu, lens=(30, 40), table=table):
        out = torch.full_like(q, 5.0)
        kvq.kvq_paged_attend(q, cache, cu, torch.tensor(lens, **dev), table, max_q_len=max(news),
                             out=out)
        return out, kvq.kvq_device_status()
    good, st = call()
    assert st == 0
    out, st = call(lens=(0, 40))  # tokens before position 0
    assert st == 0 and (out[:news[0]] == 0).all() and torch.equal(out[news[0]:], good[news[0]:])
    for lens in ((-1, 40), (49, 40)):
        out, st = call(lens=lens)
        assert st == 11 and (out[:news[0]] == 5).all() and torch.equal(out[news[0]:], good[news[0]:])
    for a in (-3, news[0] + 1, n + 2):  # not non-decreasing, or past the tokens
        out, st = call(cu=torch.tensor([a, news[0], n], **dev))
        assert st == 11 and torch.equal(out[news[0]:], good[news[0]:])
    out, st = call(cu=torch.tensor([0, news[0], n + 1], **dev))
    assert st == 11 and torch.equal(out[:news[0]], good[:news[0]])
    for bad in (-1, 8, 2 ** 31 - 1):
        t = table.clone()
        t[0, 0] = bad
        out, st = call(table=t)
        assert st == 11 and torch.equal(out[news[0]:], good[news[0]:])
        ref = O.attend_paged(np64(q), *(x.cpu().numpy() for x in cache.tensors()[:4]), cu.tolist(),
                             [30, 40], t.cpu().numpy(), cache.signs.cpu().numpy(), 0, 128, d ** -0.5)
        assert np.abs(np64(out) - ref)[:news[0]].max() < 2e-2 * np.abs(ref).max()
    t = table.clone()
    t[0, :] = -1  # every page of a sequence
    out, st = call(table=t)
    assert st == 11 and (out[:news[0]] == 0).all() and torch.equal(out[news[0]:], good[news[0]:])


def attend_f64(q, cache, cu, lens, table, window=0):
    """O.attend_paged on the GPU, for sizes the oracle is too slow for: its own
    rotation matrix, float64 throughout.  Also sum_t p_t |V_t| and the largest
    sm_scale |q| |K_t| of each (token, head)."""
    R = torch.from_numpy(O.rotation_matrix(cache.d, cache.rot)).cuda()
    R = R * cache.signs.double()
    nq = q.shape[1] // cache.n_kv_heads
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mass, far = torch.zeros_like(out[..., 0]), torch.zeros_like(out[..., 0])

    def values(packed, scales, pages, n):
        p = packed[pages].transpose(0, 1).flatten(1, 2)[:, :n].to(torch.int16)
        c = torch.stack([p & 15, p >> 4], -1).flatten(-2)
        c = torch.where(c > 7, c - 16, c).double()
        s = scales[pages].transpose(0, 1).flatten(1, 2)[:, :n].double()
        return (c * s.repeat_interleave(cache.group, -1)) @ R
    for s, n in enumerate(lens):
        pages = table[s, :-(-n // cache.page_size)].long()
        k = values(cache.k_packed, cache.k_scales, pages, n)
        v = values(cache.v_packed, cache.v_scales, pages, n)
        m = cu[s + 1] - cu[s]
        at = n - m + torch.arange(m, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")
        hide = (t > at) | ((t <= at - window) if window else torch.zeros_like(t > at))
        for h in range(cache.n_kv_heads):
            x = q[cu[s]:cu[s + 1], h * nq:(h + 1) * nq].double().transpose(0, 1)
            w = (x @ k[h].T * cache.d ** -0.5).masked_fill(hide, -torch.inf).softmax(-1)
            here = (slice(cu[s], cu[s + 1]), slice(h * nq, (h + 1) * nq))
            out[here] = (w @ v[h]).transpose(0, 1)
            mass[here] = (w @ v[h].norm(dim=-1)).T
            far[here] = (x.norm(dim=-1) * k[h].norm(dim=-1).max() * cache.d ** -0.5).T
    return out, mass, far


def check_large(kvq, cache, q, cu, lens, table, window=0):
    """By the 2-norm of each row.  Few rows: rounding the result, u, and as much
    again twice for what is before it (15-bit queries, 23-bit weights).  Chunks:
    |ds_t| <= D = 3 2^-12 sm_scale |q| |y_K,t| (a query, a ratio of scales and
    their product with a code, each rounded to 11 bits), so u |out| and
    expm1(2 D) + 2^-10 of sum_t p_t |V_t|."""
    dev = dict(device="cuda", dtype=torch.int32)
    most = max(b - a for a, b in zip(cu, cu[1:]))
    got = kvq.kvq_paged_attend(q, cache, torch.tensor(cu, **dev), torch.tensor(lens, **dev), table,
                               max_q_len=most, window=window)
    assert kvq.kvq_device_status() == 0
    ref, mass, far = attend_f64(q, cache, cu, lens, table, window)
    err = (got.double() - ref).norm(dim=-1)
    u = UNIT[q.dtype]
    if most == 1:
        assert (err <= 3 * u * ref.norm(dim=-1)).all(), (err / ref.norm(dim=-1)).max().item()
    else:
        tol = u * ref.norm(dim=-1) + (torch.expm1(6 * 2.0 ** -12 * far) + 2.0 ** -10) * mass
        assert (err <= tol).all(), (err / tol).max().item()
    # and on the whole, where the errors of many rows do not add up: 4 u
    assert err.square().sum().sqrt() <= 4 * u * ref.norm()


@pytest.mark.parametrize("d,group,nq,heads,page,seqs,length", [
    (64, 64, 1, 32, 16, 10, 16000), (64, 32, 3, 32, 64, 6, 9000), (128, 32, 4, 16, 32, 12, 8000),
    (128, 128, 8, 16, 16, 10, 6000), (256, 256, 4, 16, 64, 8, 5000), (256, 32, 8, 8, 16, 8, 5000)])
def test_attend_one_token_long(kvq, d, group, nq, heads, page, seqs, length):
    """Runs of many tiles and of several items in every block."""
    lens = [max(1, length * (s + 1) // seqs - s) for s in range(seqs)]
    cache = make_pool(kvq, d, sum(-(-m // page) for m in lens), heads, page, d, group, 0)
    table = make_batch(cache, 17, lens)
    q = rows(gen(18), seqs, heads * nq, d, torch.float16) * 0.25
    check_large(kvq, cache, q, list(range(seqs + 1)), lens, table)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("d,group,nq,heads,page,news,lens,window", [
    (64, 64, 1, 16, 16, [3000, 700], [5000, 700], 0), (64, 32, 3, 4, 64, [2500], [9001], 0),
    (128, 32, 4, 4, 32, [1500, 1, 333], [4000, 5000, 350], 0), (128, 128, 4, 4, 64, [4000], [4000], 0),
    (256, 256, 4, 2, 64, [2000, 900], [6000, 900], 512), (256, 64, 2, 4, 16, [1777], [3000], 0)])
def test_attend_chunk_long(kvq, dtype, d, group, nq, heads, page, news, lens, window):
    cache = make_pool(kvq, d, sum(-(-m // page) for m in lens), heads, page, d, group, 0)
    table = make_batch(cache, 19, lens)
    cu = np.concatenate([[0], np.cumsum(news)]).tolist()
    q = rows(gen(20), cu[-1], heads * nq, d, dtype) * 0.25
    check_large(kvq, cache, q, cu, lens, table, window)


@pytest.mark.parametrize("d,group,nq,new", [(256, 256, 6, 5), (256, 256, 8, 16), (128, 32, 8, 16),
                                            (64, 64, 4, 40), (128, 128, 4, 1), (64, 64, 1, 1)])
def test_attend_repeats(kvq, d, group, nq, new):
    """The same call many times over, runs of many tiles and items in every
    block: the roles of a block meet in ever other orders, the result stays."""
    seqs, length, heads, page = 32, 3000, 8, 32
    cache = make_pool(kvq, d, seqs * 94, heads, page, d, group, 0)
    table = make_batch(cache, 21, [length] * seqs)
    q = rows(gen(22), seqs * new, heads * nq, d, torch.float16) * 0.25
    dev = dict(device="cuda", dtype=torch.int32)
    cu = torch.arange(seqs + 1, **dev) * new
    lens = torch.full((seqs,), length, **dev)
    first = kvq.kvq_paged_attend(q, cache, cu, lens, table, max_q_len=new)
    out = torch.empty_like(first)
    for i in range(500):
        kvq.kvq_paged_attend(q, cache, cu, lens, table, max_q_len=new, out=out)
        if i % 100 == 99:
            assert kvq.kvq_device_status() == 0 and torch.equal(out, first)


def test_attend_many_sequences(kvq):
    """More sequences than threads of a block, most of them idle."""
    n = 1500
    cache = make_pool(kvq, 7, 64, 1, 16, 64, 32, 0)
    lens = [(s * 7) % 16 + 1 if s % 50 == 0 else 0 for s in range(n)]
    cu = [0]
    for s in range(n):
        cu.append(cu[-1] + (1 if s % 50 == 0 else 0))
    table = torch.arange(n, device="cuda", dtype=torch.int32)[:, None] // 50 % 64
    q = rows(gen(16), cu[-1], 2, 64, torch.float16) * 0.25
    run_attend(kvq, cache, q, cu, lens, table.contiguous())


# ------------------------------------------------------------------ together ---

@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("d,group,nq,window", [(64, 64, 1, 0), (128, 32, 6, 0), (256, 256, 4, 60)])
def test_steps_of_a_layer(kvq, dtype, d, group, nq, window):
    """A layer as a serving loop runs it: chunks of two prompts, then decoding
    steps with one of them drafting; every step checked against the oracle on
    the keys and values as the cache holds them."""
    heads, page = 2, 16
    signs = torch.from_numpy(W.make_signs(d)).cuda()
    cache = kvq.PagedCache.empty(40, heads, page, d, group, signs)
    table = torch.randperm(40, generator=gen(1), device="cuda").to(torch.int32).reshape(2, 20)
    rope = kvq.rope_table(400, d)
    g = gen(d + nq)
    qw, kw = (1 + 0.1 * torch.randn(d, generator=g, device="cuda") for _ in range(2))
    lens = [0, 0]
    for news in ([100, 37], [60, 0], [1, 1], [4, 1], [1, 1], [1, 1]):
        lens = [a + b for a, b in zip(lens, news)]
        n = sum(news)
        qkv = rows(g, n, heads * (nq + 2), d, dtype)
        q, k, v = qkv.split([heads * nq, heads, heads], 1)
        cu_t = torch.tensor([0, news[0], n], device="cuda", dtype=torch.int32)
        len_t = torch.tensor(lens, device="cuda", dtype=torch.int32)
        pos, slots = kvq.paged_rows(cu_t, len_t, table, page, n)
        kvq.kvq_paged_append(k, v, slots, cache, positions=pos, cos_sin=rope, k_weight=kw)
        kvq.kvq_qk_norm_rope(q, positions=pos, cos_sin=rope, q_weight=qw, q_out=q)
        want = O.norm_rope(np64(k), np64(kw), pos.tolist(), rope.cpu().numpy())
        check_append(kvq, cache, slots, (want, np64(v)), (None, None), dtype)
        run_attend(kvq, cache, q, [0, news[0], n], lens, table, window=window)


# ----------------------------------------------------- streams, graphs, devices ---

def layer_state(kvq, d, group, news, seed, dtype=torch.float16):
    """A batch in flight: cache with history, new tokens, tables."""
    heads, nq, page = 2, 4, 16
    signs = torch.from_numpy(W.make_signs(d)).cuda()
    cache = make_pool(kvq, seed, 40, heads, page, d, group, 0)
    lens = [150 + n for n in news]
    table = torch.randperm(40, generator=gen(seed), device="cuda").to(torch.int32).reshape(2, 20)
    n = sum(news)
    qkv = rows(gen(seed + 1), n, heads * (nq + 2), d, dtype)
    dev = dict(device="cuda", dtype=torch.int32)
    cu, ln = torch.tensor([0, news[0], n], **dev), torch.tensor(lens, **dev)
    pos, slots = kvq.paged_rows(cu, ln, table, page, n)
    return dict(cache=cache, qkv=qkv, cu=cu, ln=ln, table=table, pos=pos, slots=slots,
                rope=kvq.rope_table(400, d), most=max(news), nq=heads * nq, heads=heads,
                w=1 + 0.1 * torch.randn(d, generator=gen(seed + 2), device="cuda"))


def layer(kvq, s, stream=None):
    q, k, v = s["qkv"].split([s["nq"], s["heads"], s["heads"]], 1)
    kvq.kvq_paged_append(k, v, s["slots"], s["cache"], positions=s["pos"], cos_sin=s["rope"],
                         k_weight=s["w"], stream=stream)
    q, _ = kvq.kvq_qk_norm_rope(q, positions=s["pos"], cos_sin=s["rope"], q_weight=s["w"],
                                stream=stream)
    return kvq.kvq_paged_attend(q, s["cache"], s["cu"], s["ln"], s["table"], max_q_len=s["most"],
                                stream=stream)


LAYERS = [(64, 64, [1, 1]), (128, 32, [3, 1]), (256, 256, [40, 7]), (128, 128, [90, 60])]


@pytest.mark.parametrize("d,group,news", LAYERS)
def test_captured_layer_replays(kvq, d, group, news):
    """A layer captured into a graph follows what its inputs hold at each
    replay: other tokens, other lengths, other pages."""
    s, other = layer_state(kvq, d, group, news, 3), layer_state(kvq, d, group, news, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        out = layer(kvq, s)
    torch.cuda.current_stream().wait_stream(side)
    for x in (s, other):
        # (the graph's inputs take x's values; x itself is computed eagerly on copies)
        eager = dict(x, cache=kvq.PagedCache(*(t.clone() for t in x["cache"].tensors()), 0))
        want = layer(kvq, eager)
        if x is other:
            for name in ("qkv", "cu", "ln", "table", "pos", "slots", "w"):
                s[name].copy_(x[name])
            for a, b in zip(s["cache"].tensors(), x["cache"].tensors()):
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for a, b in zip(s["cache"].tensors(), eager["cache"].tensors()):
            assert torch.equal(a, b)
    assert kvq.kvq_device_status() == 0
    del graph


def test_two_streams_at_once(kvq):
    """Calls of different shapes on two streams, each its own workspace: the
    results are those of calls one after the other."""
    states = [layer_state(kvq, d, g, n, 10 + i) for i, (d, g, n) in enumerate(LAYERS)]
    want = [layer(kvq, s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(20):
        got = [layer(kvq, s, stream=st) for s, st in zip(states, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    assert kvq.kvq_device_status() == 0
    # a raw handle, and a stream that is current
    got = layer(kvq, states[1], stream=streams[0].cuda_stream)
    streams[0].synchronize()
    assert torch.equal(got, want[1])
    with torch.cuda.stream(streams[2]):
        got = layer(kvq, states[2])
    streams[2].synchronize()
    assert torch.equal(got, want[2])


def test_own_workspace_and_refusals(kvq):
    s = layer_state(kvq, 128, 32, [3, 1], 5)
    want = layer(kvq, s)
    q, k, v = s["qkv"].split([s["nq"], s["heads"], s["heads"]], 1)
    q, _ = kvq.kvq_qk_norm_rope(q, positions=s["pos"], cos_sin=s["rope"], q_weight=s["w"])
    need = kvq.lib.kvq_paged_attend_workspace(q.shape[0], s["heads"], 4, 128, s["most"])
    args = (q, s["cache"], s["cu"], s["ln"], s["table"])
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # holds no meaning before
    assert torch.equal(kvq.kvq_paged_attend(*args, max_q_len=s["most"], workspace=ws), want)
    with pytest.raises(kvq.KVQError, match="BAD_SIZE"):
        kvq.kvq_paged_attend(*args, max_q_len=s["most"], workspace=ws[:-256])
    with pytest.raises(kvq.KVQError, match="MISALIGNED"):
        kvq.kvq_paged_attend(*args, max_q_len=s["most"], workspace=torch.cat([ws, ws])[16:])
    with pytest.raises(ValueError, match="does not fit"):
        kvq.kvq_paged_attend(q[:, :7], *args[1:], max_q_len=1)
    with pytest.raises(ValueError, match="contiguous"):
        kvq.kvq_paged_attend(q[..., ::2].repeat(1, 1, 2)[:, ::2], *args[1:], max_q_len=1)
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        kvq.kvq_paged_attend(q.float(), *args[1:], max_q_len=1)
    with pytest.raises(TypeError, match="int32"):
        kvq.kvq_paged_attend(q, s["cache"], s["cu"].long(), *args[3:], max_q_len=1)
    with pytest.raises(ValueError, match="positions"):
        kvq.kvq_qk_norm_rope(q, cos_sin=s["rope"])
    with pytest.raises(TypeError, match="bfloat16"):
        kvq.kvq_paged_append(k.bfloat16(), v, s["slots"], s["cache"])
    with pytest.raises(kvq.KVQError, match="MISALIGNED"):
        wide = torch.zeros((4, 9 * 128 + 8), dtype=torch.float16, device="cuda")
        kvq.kvq_qk_norm_rope(wide[:, 4:4 + 8 * 128].unflatten(1, (8, 128)))
    with pytest.raises(kvq.KVQError, match="BAD_SIZE"):  # a token stride that is no multiple of 8
        wide = torch.zeros((4, 8 * 128 + 4), dtype=torch.float16, device="cuda")
        kvq.kvq_qk_norm_rope(wide[:, :8 * 128].unflatten(1, (8, 128)))


def test_no_tokens_and_no_sequences(kvq):
    s = layer_state(kvq, 64, 32, [2, 1], 6)
    q = s["qkv"][:, :s["nq"]]
    none = kvq.kvq_paged_attend(q[:0], s["cache"], s["cu"] * 0, s["ln"], s["table"], max_q_len=1)
    assert none.shape == (0, s["nq"], 64)
    out = torch.full_like(q, 3.0)
    kvq.kvq_paged_attend(q, s["cache"], s["cu"][:1], s["ln"][:0], s["table"][:0], max_q_len=1, out=out)
    kvq.kvq_paged_attend(q, s["cache"], s["cu"] * 0, s["ln"], s["table"], max_q_len=1, out=out)
    assert (out == 3.0).all()  # tokens of no sequence
    kvq.kvq_paged_append(q[:0, :2], q[:0, :2], s["slots"][:0], s["cache"])
    assert kvq.kvq_device_status() == 0
