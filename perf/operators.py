"""Cases of the paged-cache operators: query/key norm with position rotation, appending
new keys and values to the paged int4 cache, and attention of new tokens over that cache.

``run`` computes each operator in its plain form (elementary torch operations, 32 bits)
or, with ``own`` set, through the package's entry points; ``exact`` evaluates the
definitions in 64 bits.  The definitions:

* norm and rotation, for a row x of d values at position p:
      n = x / sqrt(mean(x^2) + eps) * weight                  (left out without a weight)
      pairs (a, b) = (n[i], n[i + r/2]), or (n[2i], n[2i + 1]) when interleaved, i < r/2:
      (a cos - b sin, a sin + b cos) of the table row p;  values from r on pass through.
* forward step: y = R D x, per group of g values s = max|y| / 7, code = round(y / s);
  a cached row stands for D R^T (s code), D = diag(signs), R the packed real Fourier
  transform (rot 0) or the Walsh-Hadamard transform (rot 1).
* attention: the i-th of a sequence's n new tokens stands at position p = len - n + i and
  attends the cached rows t with p - window < t <= p (window 0: all t <= p).
"""

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
THETA = 10000.0


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # One decoded token of a Gemma-3-1B-like layer: 4 query heads and 1 key head.
        dict(name="norm_rope one token", op="norm_rope", tokens=1, heads=4, kv_heads=1, d=256,
             rot_dim=256, norm=True, interleaved=False, dtype="bf16"),
        # A prefill chunk of odd length, Qwen2.5-1.5B-like heads (12 and 2).
        dict(name="norm_rope chunk", op="norm_rope", tokens=1021, heads=12, kv_heads=2, d=128,
             rot_dim=64, norm=True, interleaved=True, dtype="f16"),
        # A long prefill, SmolLM2-1.7B-like heads, rotation only.
        dict(name="norm_rope prefill", op="norm_rope", tokens=8192, heads=32, kv_heads=32, d=64,
             rot_dim=64, norm=False, interleaved=False, dtype="bf16"),
        # One new token for each of 16 sequences, SmolLM2-1.7B-like cache.
        dict(name="append decode", op="append", tokens=16, kv_heads=32, d=64, group=64, rot=0,
             page=16, rot_dim=64, norm=False, interleaved=False, dtype="f16"),
        # A prefill chunk into a cache with one scale per 32 values.
        dict(name="append chunk", op="append", tokens=2045, kv_heads=2, d=128, group=32, rot=0,
             page=32, rot_dim=128, norm=True, interleaved=False, dtype="bf16"),
        # A long prefill.
        dict(name="append prefill", op="append", tokens=16384, kv_heads=8, d=128, group=128, rot=0,
             page=64, rot_dim=128, norm=True, interleaved=False, dtype="bf16"),
        # One decoded token of a Gemma-3-1B-like layer, where latency counts.
        dict(name="attend one token", op="attend", seqs=1, new=1, longest=4096, ragged=False,
             kv_heads=1, queries=4, d=256, group=256, rot=0, page=64, window=0, dtype="bf16"),
        # A decoding batch: 16 long SmolLM2-1.7B-like sequences.
        dict(name="attend decode d64", op="attend", seqs=16, new=1, longest=16384, ragged=False,
             kv_heads=32, queries=1, d=64, group=64, rot=0, page=16, window=0, dtype="f16"),
        # A decoding batch of 64 sequences of all lengths, one scale per 32 values.
        dict(name="attend decode d128", op="attend", seqs=64, new=1, longest=8192, ragged=True,
             kv_heads=8, queries=4, d=128, group=32, rot=0, page=32, window=0, dtype="bf16"),
        # A few drafted tokens for each sequence, checked in one pass.
        dict(name="attend drafted", op="attend", seqs=8, new=5, longest=2048, ragged=True,
             kv_heads=2, queries=6, d=128, group=32, rot=0, page=16, window=0, dtype="f16"),
        # A chunk of a long prompt over what is cached of it.
        dict(name="attend chunk", op="attend", seqs=1, new=4096, longest=16384, ragged=False,
             kv_heads=8, queries=4, d=128, group=128, rot=0, page=64, window=0, dtype="bf16"),
        # Ragged chunks of a Gemma-3-1B-like layer with a sliding window.
        dict(name="attend window", op="attend", seqs=4, new=2000, longest=8000, ragged=True,
             kv_heads=1, queries=4, d=256, group=256, rot=0, page=64, window=512, dtype="f16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "attend", "attend"])
    d = rng.choice([64, 128, 256])
    dtype = rng.choice(["f16", "bf16"])
    rope = dict(rot_dim=rng.choice([d, d, d // 2]), norm=rng.random() < 0.5,
                interleaved=rng.random() < 0.3, dtype=dtype)
    group = rng.choice([g for g in (32, 64, 128, 256) if g <= d] + [d])
    cache = dict(d=d, group=group, rot=rng.choice([0, 0, 1]), page=rng.choice([16, 32, 64, 128]))
    if op == "norm_rope":
        kv = rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_log(rng, 1, 8192 * 32 * 64 // (12 * kv * d)),
                    heads=kv * rng.choice([1, 3, 4, 8]), kv_heads=kv, d=d, **rope)
    if op == "append":
        kv = rng.choice([1, 2, 5, 8])
        return dict(op=op, tokens=_log(rng, 1, 16384 * 128 // d * 8 // kv // 2), kv_heads=kv,
                    **cache, **rope)
    kv, queries = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8])
    if rng.random() < 0.5:  # decoding, a few tokens at most
        seqs, longest = _log(rng, 1, 48), _log(rng, 1, 8192)
        new = rng.choice([1, 1, 1, 2, 4])
    else:  # chunks
        seqs, longest = rng.choice([1, 1, 2, 3]), _log(rng, 200, 8192)
        new = _log(rng, 16, 1024)
    return dict(op=op, seqs=seqs, new=min(new, longest), longest=longest, ragged=rng.random() < 0.6,
                kv_heads=kv, queries=queries, window=rng.choice([0, 0, 300]), dtype=dtype, **cache)


def _lengths(case):
    """(new tokens, cached rows) of every sequence of an attend case; the first is the longest."""
    new, length = [], []
    for s in range(case["seqs"]):
        part = 1.0 if s == 0 or not case["ragged"] else ((s * 0.61803398875) % 1.0)
        n = max(1, int(round(case["new"] * (part if case["new"] > 8 else 1.0))))
        new.append(n)
        length.append(max(n, int(round(case["longest"] * part))))
    return new, length


# ----------------------------------------------------------------- inputs ---

def _rotation(d, rot):
    """R in 64 bits, row k the k-th rotated coordinate."""
    n = torch.arange(d, dtype=torch.int64)
    if rot == 1:
        both = n[:, None] & n[None, :]
        odd = torch.zeros_like(both)
        for b in range(8):
            odd ^= (both >> b) & 1
        return (1 - 2 * odd).double() / math.sqrt(d)
    k = torch.arange(1, d // 2, dtype=torch.int64)
    turn = (k[:, None] * n[None, :]) % d
    angle = turn.double() * (2 * math.pi / d)
    R = torch.empty((d, d), dtype=torch.float64)
    R[0], R[1] = 1.0, (1 - 2 * (n % 2)).double()
    R[2::2], R[3::2] = math.sqrt(2) * torch.cos(angle), -math.sqrt(2) * torch.sin(angle)
    return R / math.sqrt(d)


def _table(n_pos, rot_dim):
    inv = THETA ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device="cuda") / rot_dim)
    angle = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _channels(gen, heads, d):
    """Factors of the channels of each head: a few are many times the others."""
    f = torch.ones((heads, d), device="cuda")
    at = torch.rand((heads, d), generator=gen, device="cuda").argsort(1)[:, :4]
    return f.scatter_(1, at, 10.0 + 10.0 * torch.rand((heads, 4), generator=gen, device="cuda"))


def _heads(gen, tokens, heads, d, dtype):
    x = torch.randn((tokens, heads, d), generator=gen, device="cuda")
    return (x * _channels(gen, heads, d)).to(DTYPES[dtype])


def _fill(gen, pages, heads, page, d, group, signs, R):
    """Codes and scales of a cache whose pages all hold rows of a model's keys or values."""
    packed = torch.empty((pages, heads, page, d // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, heads, page, d // group), device="cuda")
    factor = _channels(gen, heads, d)[None, :, None, :] * signs
    step = max(1, (1 << 26) // (heads * page * d))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = torch.randn((n, heads, page, d), generator=gen, device="cuda") * factor
        y = (x @ R.t()).view(n, heads, page, d // group, group)
        s = y.abs().amax(-1) / 7
        q = (y / s[..., None]).round_().to(torch.int8).view(n, heads, page, d) & 15
        packed[a:a + n] = (q[..., 0::2] | (q[..., 1::2] << 4)).view(torch.uint8)
        scales[a:a + n] = s
    return packed, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, d = case["op"], case["d"]
    st = dict(case)
    if op == "norm_rope":
        t, far = case["tokens"], 32768
        # a model's fused projection: queries, keys and values of a token lie side by side
        h, kv = case["heads"], case["kv_heads"]
        qkv = _heads(gen, t, h + 2 * kv, d, case["dtype"])
        st.update(q=qkv[:, :h], k=qkv[:, h:h + kv], table=_table(far, case["rot_dim"]))
        first = int(torch.randint(0, far - t, (1,), generator=gen, device="cuda"))
        st["positions"] = torch.arange(first, first + t, device="cuda", dtype=torch.int32)
        for name in ("q_weight", "k_weight"):
            st[name] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda") if case["norm"] else None
        return st
    signs = torch.where(torch.rand(d, generator=gen, device="cuda") < 0.5, -1, 1).to(torch.int8)
    R = _rotation(d, case["rot"]).float().cuda()
    st.update(signs=signs, R=R)
    page, kv, g = case["page"], case["kv_heads"], case["group"]
    if op == "append":
        t = case["tokens"]
        pages = t // page + 2
        order = torch.randperm(pages, generator=gen, device="cuda")
        at = torch.arange(t, device="cuda") + page // 2  # starts inside a page
        qkv = _heads(gen, t, 2 * kv, d, case["dtype"])
        st.update(k=qkv[:, :kv], v=qkv[:, kv:], slots=order[at // page] * page + at % page,
                  positions=(at + 1000).to(torch.int32), table=_table(t + page + 1000, case["rot_dim"]),
                  k_weight=1 + 0.2 * torch.randn(d, generator=gen, device="cuda") if case["norm"] else None)
        for name in ("k", "v"):
            st[name + "_packed"] = torch.zeros((pages, kv, page, d // 2), dtype=torch.uint8, device="cuda")
            st[name + "_scales"] = torch.zeros((pages, kv, page, d // g), device="cuda")
            st[name + "_hat"] = torch.zeros((t, kv, d), dtype=DTYPES[case["dtype"]], device="cuda")
        return st
    new, length = _lengths(case)
    need = [-(-n // page) for n in length]
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    rows = torch.zeros((case["seqs"], max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        rows[s, :n] = order[at:at + n]
        at += n
    st["page_table"] = rows
    total = sum(new)
    h = kv * case["queries"]
    st["q"] = torch.randn((total, h, d), generator=gen, device="cuda").to(DTYPES[case["dtype"]])
    ends = [0]
    for n in new:
        ends.append(ends[-1] + n)
    st["cu_q"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    st["kv_len"] = torch.tensor(length, dtype=torch.int32, device="cuda")
    st["max_new"], st["max_len"] = max(new), max(length)
    for name in ("k", "v"):
        st[name + "_packed"], st[name + "_scales"] = _fill(gen, pages, kv, page, d, g, signs, R)
    return st


# -------------------------------------------------------------- plain forms ---

def _norm_rope(x, weight, positions, table, interleaved, eps=1e-6):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight
    half = table.shape[1] // 2
    row = table[positions.long()][:, None, :]
    c, s = row[..., :half], row[..., half:]
    if interleaved:
        a, b, rest = x[..., 0:2 * half:2], x[..., 1:2 * half:2], x[..., 2 * half:]
        turned = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
        return torch.cat([turned, rest], -1)
    a, b, rest = x[..., :half], x[..., half:2 * half], x[..., 2 * half:]
    return torch.cat([a * c - b * s, a * s + b * c, rest], -1)


def _append(st, name, x):
    t, h, d = x.shape
    g, page = st["group"], st["page"]
    y = ((x * st["signs"]) @ st["R"].t()).view(t, h, d // g, g)
    s = y.abs().amax(-1) / 7
    q = torch.where(s[..., None] > 0, y / s[..., None], 0).round().clamp(-8, 7)
    code = q.to(torch.int8).view(t, h, d) & 15
    at, off = st["slots"] // page, st["slots"] % page
    st[name + "_packed"][at, :, off] = (code[..., 0::2] | (code[..., 1::2] << 4)).view(torch.uint8)
    st[name + "_scales"][at, :, off] = s
    hat = ((q * s[..., None]).view(t, h, d) @ st["R"]) * st["signs"]
    st[name + "_hat"].copy_(hat)


def _rows(st, name):
    """The rotated rows [seqs, heads, length, d] that the cache holds, in 32 bits."""
    codes = st[name + "_packed"][st["page_table"].long()].transpose(1, 2).flatten(2, 3)
    scales = st[name + "_scales"][st["page_table"].long()].transpose(1, 2).flatten(2, 3)
    codes, scales = codes[:, :, :st["max_len"]], scales[:, :, :st["max_len"]]
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).to(torch.int8)
    y = ((both ^ 8) - 8).float().unflatten(-1, (-1, st["group"]))
    return (y * scales[..., None]).flatten(-2)


def _attend(st):
    total, h, d = st["q"].shape
    kv, page = st["kv_heads"], st["page"]
    start, length = st["cu_q"][:-1].long(), st["kv_len"].long()
    new = st["cu_q"][1:].long() - start
    i = torch.arange(st["max_new"], device="cuda")
    here = i < new[:, None]  # [seqs, new]
    token = torch.where(here, start[:, None] + i, 0)
    q = ((st["q"].float() * st["signs"]) @ st["R"].t())[token]  # [seqs, new, heads, d]
    q = q.unflatten(2, (kv, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores = (q @ _rows(st, "k").transpose(2, 3)).mul_(d ** -0.5)
    at = (length[:, None] - new[:, None] + i)[:, :, None]
    t = torch.arange(st["max_len"], device="cuda")
    seen = (t <= at) & (t < length[:, None, None]) & here[:, :, None]
    if st["window"]:
        seen &= t > at - st["window"]
    seen = seen.repeat_interleave(h // kv, 1)[:, None]
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top.isfinite(), top, 0)).exp_()
    norm = p.sum(-1, keepdim=True)
    o = (p @ _rows(st, "v")) / torch.where(norm > 0, norm, 1)
    o = (o @ st["R"]) * st["signs"]
    o = o.unflatten(2, (-1, h // kv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return o[here].to(st["q"].dtype)


def run(st):
    if own:
        from rotated_int4_kv_kvq_b200 import kvq
        if st["op"] == "norm_rope":
            return kvq.kvq_qk_norm_rope(st["q"], st["k"], positions=st["positions"],
                                        cos_sin=st["table"], interleaved=st["interleaved"],
                                        q_weight=st["q_weight"], k_weight=st["k_weight"], eps=1e-6)
        cache = kvq.PagedCache(st["k_packed"], st["k_scales"], st["v_packed"], st["v_scales"],
                               st["signs"], st["rot"])
        if st["op"] == "append":
            kvq.kvq_paged_append(st["k"], st["v"], st["slots"], cache, positions=st["positions"],
                                 cos_sin=st["table"], interleaved=st["interleaved"],
                                 k_weight=st["k_weight"], eps=1e-6, k_hat=st["k_hat"],
                                 v_hat=st["v_hat"])
            return st["k_hat"], st["v_hat"], st["k_scales"], st["v_scales"]
        return kvq.kvq_paged_attend(st["q"], cache, st["cu_q"], st["kv_len"], st["page_table"],
                                    max_q_len=st["max_new"], window=st["window"])
    if st["op"] == "norm_rope":
        return tuple(_norm_rope(st[n], st[n + "_weight"], st["positions"], st["table"],
                                st["interleaved"]).to(st[n].dtype) for n in ("q", "k"))
    if st["op"] == "append":
        _append(st, "k", _norm_rope(st["k"], st["k_weight"], st["positions"], st["table"],
                                    st["interleaved"]))
        _append(st, "v", st["v"].float())
        return st["k_hat"], st["v_hat"], st["k_scales"], st["v_scales"]
    return _attend(st)


# -------------------------------------------------------------------- work ---

def work(case):
    d = case["d"]
    if case["op"] == "norm_rope":
        n = case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": n * d * 4 + case["tokens"] * (case["rot_dim"] * 4 + 4),
                "flops": n * (3 * case["rot_dim"] + (4 * d if case["norm"] else 0))}
    row = d // 2 + 4 * (d // case["group"])
    if case["op"] == "append":
        n = case["tokens"] * case["kv_heads"] * 2  # rows in, codes and scales out, dequantized out
        return {"bytes": n * (4 * d + row) + case["tokens"] * (case["rot_dim"] * 4 + 12),
                "flops": n * 2 * 2.5 * d * math.log2(d)}
    rows = pairs = 0
    for n, length in zip(*_lengths(case)):
        w = case["window"] or length
        first = max(0, length - n - w + 1)
        rows += length - first
        # row i attends min(position + 1, w) rows
        a, b = length - n + 1, length  # the smallest and the largest position + 1
        low = max(0, min(b, w) - a + 1)
        pairs += low * (2 * a + low - 1) // 2 + (n - low) * w
    new, _ = _lengths(case)
    h = case["kv_heads"] * case["queries"]
    return {"bytes": rows * case["kv_heads"] * 2 * row + sum(new) * h * d * 4, "flops": 4 * d * h * pairs}


# ------------------------------------------------------------------- exact ---

def _turned(x, weight, positions, table, interleaved):
    """Norm and rotation in 64 bits, as complex products."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
    r = table.shape[1]
    row = table.double()[positions.long()]
    turn = torch.complex(row[:, :r // 2], row[:, r // 2:])[:, None]
    out = x.clone()
    if interleaved:
        z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2)) * turn
        out[..., :r] = torch.view_as_real(z).reshape(*x.shape[:-1], r)
    else:
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous()) * turn
        out[..., :r // 2], out[..., r // 2:r] = z.real, z.imag
    return out


def _values(st, name, pages):
    """Rows D R^T (s code) of the given pages of every head, in 64 bits: [heads, rows, d]."""
    p = st[name + "_packed"][pages].to(torch.int32)
    c = torch.empty((*p.shape[:-1], st["d"]), dtype=torch.float64, device="cuda")
    c[..., 0::2] = ((p % 16 + 8) % 16 - 8).double()
    c[..., 1::2] = ((p // 16 + 8) % 16 - 8).double()
    c *= st[name + "_scales"][pages].double().repeat_interleave(st["group"], -1)
    x = c @ _rotation(st["d"], st["rot"]).cuda() * st["signs"].double()
    return x.transpose(0, 1).reshape(st["kv_heads"], -1, st["d"])


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rope":
        return tuple(_turned(st[n], st[n + "_weight"], st["positions"], st["table"],
                             case["interleaved"]) for n in ("q", "k"))
    d, g, page = case["d"], case["group"], case["page"]
    if case["op"] == "append":
        R = _rotation(d, case["rot"]).cuda()
        hats, scales = [], []
        for n in ("k", "v"):
            x = st[n].double() if n == "v" else _turned(st[n], st["k_weight"], st["positions"],
                                                        st["table"], case["interleaved"])
            y = torch.einsum("thj,kj->thk", x * st["signs"].double(), R)
            y = y.reshape(*y.shape[:2], d // g, g)
            s = y.abs().max(-1).values / 7
            hat = (torch.round(y / s[..., None]) * s[..., None]).reshape(*y.shape[:2], d)
            hats.append(torch.einsum("thk,kj->thj", hat, R) * st["signs"].double())
            all_s = st[n + "_scales"].double()
            flat = all_s.transpose(1, 2).contiguous().reshape(-1, s.shape[1], s.shape[2])  # by slot
            flat[st["slots"]] = s
            scales.append(flat.reshape(all_s.shape[0], page, *s.shape[1:]).transpose(1, 2).contiguous())
        return (*hats, *scales)
    new, length = _lengths(case)
    if sum(n * m for n, m in zip(new, length)) * case["kv_heads"] * case["queries"] * d > 4e12:
        return None
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    nq, at = case["queries"], 0
    for s, (n, m) in enumerate(zip(new, length)):
        pages = st["page_table"][s, :-(-m // page)].long()
        k, v = _values(st, "k", pages)[:, :m], _values(st, "v", pages)[:, :m]
        back = torch.arange(m, device="cuda") - (m - n + torch.arange(n, device="cuda"))[:, None]
        hidden = back > 0
        if case["window"]:
            hidden = hidden | (back <= -case["window"])
        for h in range(case["kv_heads"]):
            q = st["q"][at:at + n, h * nq:(h + 1) * nq].double()
            w = torch.einsum("nqd,md->qnm", q, k[h]) / math.sqrt(d)
            w = torch.softmax(w.masked_fill(hidden, -math.inf), -1)
            out[at:at + n, h * nq:(h + 1) * nq] = torch.einsum("qnm,md->nqd", w, v[h])
        at += n
    return out
