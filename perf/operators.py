"""Cases that measure the operators around a paged cache: the norm and rotation
of the query, probe and key heads (forward, backward, and with the cache
append in the same pass) and the attention of a chunk of new tokens over the
paged cache.

`run` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end), or, with `own` set, through the framework's
entry points. Shapes follow the library's benchmark configurations (16 query
heads over 8 kv heads of 128 dimensions, contexts of 4096 and 32768) and
smaller or odd ones of the same kind.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ cases ----
def listed():
    return [
        # training, or the prefill of a full batch: 4 sequences of 4096 tokens,
        # sliced out of one fused projection, written in the (B, H, L, D) layout
        dict(name="rope_train", op="rope", tokens=16384, seq_len=4096, Hq=16, Hkv=8, D=128,
             rot=128, dtype="bf16", interleaved=False, probe=True, r_norm=True),
        # a packed batch with an odd token count, fp32, half the dimensions
        # rotated in neighbouring pairs, no norm on the probe
        dict(name="rope_odd_f32", op="rope", tokens=1037, seq_len=0, Hq=8, Hkv=2, D=64, rot=32,
             dtype="f32", interleaved=True, probe=True, r_norm=False),
        # the same two in the backward direction
        dict(name="rope_bwd_train", op="rope_bwd", tokens=16384, seq_len=4096, Hq=16, Hkv=8,
             D=128, rot=128, dtype="bf16", interleaved=False, probe=True, r_norm=True),
        dict(name="rope_bwd_odd_f32", op="rope_bwd", tokens=777, seq_len=0, Hq=4, Hkv=4, D=64,
             rot=64, dtype="f32", interleaved=False, probe=True, r_norm=True),
        # the smallest call: one sequence's next token
        dict(name="append_one", op="append", B=1, qmax=1, kv_max=4096, ragged=False, pad=0,
             page=256, Hq=16, Hkv=8, D=128, rot=128, dtype="bf16", interleaved=False,
             probe=True, r_norm=True),
        # a decode step of a serving batch, one token each
        dict(name="append_step", op="append", B=128, qmax=1, kv_max=512, ragged=True, pad=0,
             page=64, Hq=16, Hkv=8, D=128, rot=128, dtype="bf16", interleaved=False,
             probe=True, r_norm=True),
        # prompts of odd lengths entering the cache, in a padded batch
        dict(name="append_chunks", op="append", B=12, qmax=1024, kv_max=2048, ragged=True,
             pad=37, page=256, Hq=16, Hkv=8, D=128, rot=128, dtype="bf16", interleaved=False,
             probe=True, r_norm=True),
        # a few drafted tokens of each sequence, checked at once
        dict(name="chunk_drafts", op="chunk", B=32, qmax=4, kv_max=4096, ragged=False, pad=0,
             page=256, Hq=16, Hkv=8, D=128, probe=True, causal=True, poison=False),
        # one prompt chunk over a cache of middle length
        dict(name="chunk_prompt", op="chunk", B=1, qmax=512, kv_max=8192, ragged=False, pad=0,
             page=256, Hq=16, Hkv=8, D=128, probe=True, causal=True, poison=False),
        # a mixed batch: odd chunk lengths from 1 to 512 over odd contexts, the
        # unused slots of the last pages holding NaN
        dict(name="chunk_mixed", op="chunk", B=24, qmax=512, kv_max=4096, ragged=True, pad=21,
             page=64, Hq=16, Hkv=8, D=128, probe=True, causal=True, poison=True),
        # a large chunk of a long context
        dict(name="chunk_long", op="chunk", B=1, qmax=2048, kv_max=32768, ragged=False, pad=0,
             page=256, Hq=16, Hkv=8, D=128, probe=True, causal=True, poison=False),
        # small heads in groups of four, odd sizes
        dict(name="chunk_small", op="chunk", B=3, qmax=173, kv_max=1000, ragged=True, pad=0,
             page=128, Hq=8, Hkv=2, D=64, probe=True, causal=True, poison=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "chunk", "chunk"])
    D = rng.choice([64, 128, 128])
    G = rng.choice([1, 2, 2, 4])
    Hkv = rng.choice([1, 2, 4, 8])
    probe = rng.random() < 0.8
    if op in ("rope", "rope_bwd", "append"):
        c = dict(op=op, Hq=G * Hkv, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2, 16]),
                 dtype=rng.choice(["bf16", "bf16", "f32"]), interleaved=rng.random() < 0.3,
                 probe=probe, r_norm=rng.random() < 0.6)
        if op == "append":
            one = rng.random() < 0.5
            B = _log_int(rng, 1, 128 if one else 16)
            c.update(B=B, qmax=1 if one else _log_int(rng, 2, 1024),
                     kv_max=_log_int(rng, 1, 4096 if B <= 16 else 512),
                     ragged=rng.random() < 0.7, pad=0 if one else rng.choice([0, 0, 5]),
                     page=rng.choice([64, 128, 256]))
            c["qmax"] = min(c["qmax"], c["kv_max"])
        else:
            L = _log_int(rng, 1, 4096)
            B = rng.randint(1, 4)
            c.update(tokens=B * L, seq_len=L if rng.random() < 0.5 else 0)
        return c
    kv = _log_int(rng, 1, 16384)
    B = _log_int(rng, 1, max(1, min(32, 65536 // kv)))
    q = _log_int(rng, 1, max(1, min(kv, 2048, 65536 // (B * Hkv * G))))
    return dict(op=op, B=B, qmax=q, kv_max=kv, ragged=rng.random() < 0.6, pad=rng.choice([0, 0, 3]),
                page=rng.choice([64, 128, 256]), Hq=G * Hkv, Hkv=Hkv, D=D, probe=probe,
                causal=rng.random() < 0.85, poison=rng.random() < 0.5)


# ----------------------------------------------------------------- inputs ----
def _rope_table(n, rot, base=1e6):
    """[n, rot] fp32: the cosines of n positions' angles, then the sines."""
    inv = base ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    ang = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def _lengths(c):
    """The new tokens of each sequence and its length after them: all alike, or
    a ragged batch's spread (chunks by their logarithm, lengths from a quarter
    of the longest up, none shorter than its chunk)."""
    q, kv, B = min(c["qmax"], c["kv_max"]), c["kv_max"], c["B"]
    if not c["ragged"]:
        return [q] * B, [kv] * B
    us = [(i + 0.5) / max(1, B - 1) for i in range(B - 1)]
    qs = [q] + [max(1, round(q ** u)) for u in us]
    mix = [(7 * i + 3) % max(1, B - 1) for i in range(B - 1)]  # lengths in another order
    ns = [kv] + [max(round(kv // 4 + us[m] * (kv - kv // 4)), n) for m, n in zip(mix, qs[1:])]
    return qs, ns


def _cache(c, s, host, dev, dtype):
    """Lengths, a page table over a pool in a random order, and the pool."""
    qs, ns = _lengths(c)
    B, ps = c["B"], c["page"]
    order = torch.randperm(B, generator=host).tolist()
    qs, ns = [qs[i] for i in order], [ns[i] for i in order]
    maxp = -(-max(ns) // ps)
    need = [-(-n // ps) for n in ns]
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=host)
    table = torch.zeros(B, maxp, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]].int()
        at += need[b]
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(qs).cumsum(0)
    s["qs"], s["ns"], s["total"] = qs, ns, sum(qs) + c["pad"]
    s["qmax"], s["kmax"] = max(qs), max(ns)
    s["cu"], s["lens"], s["table"] = cu.cuda(), torch.tensor(ns, dtype=torch.int32).cuda(), table.cuda()
    shape = (pages, ps, c["Hkv"], c["D"])
    s["k_pages"] = torch.randn(shape, generator=dev, device="cuda").to(dtype)
    s["v_pages"] = torch.randn(shape, generator=dev, device="cuda").to(dtype)
    if c.get("poison"):  # slots that no sequence fills
        for b in range(B):
            used = ns[b] - (need[b] - 1) * ps
            s["k_pages"][table[b, need[b] - 1], used:] = float("nan")
            s["v_pages"][table[b, need[b] - 1], used:] = float("nan")
        s["k_pages"][order[-1]] = float("nan")
        s["v_pages"][order[-1]] = float("nan")


def prepare(case, seed):
    c = case
    host = torch.Generator().manual_seed(seed)
    dev = torch.Generator(device="cuda").manual_seed(seed)
    s = {"c": c}
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "chunk":
        _cache(c, s, host, dev, torch.bfloat16)
        n = s["total"]
        s["q"] = torch.randn(n, Hq, D, generator=dev, device="cuda").bfloat16()
        s["r"] = ((torch.randn(n, Hq, D, generator=dev, device="cuda") * 0.5).bfloat16()
                  if c["probe"] else None)
        s["out"] = torch.zeros(n, Hq, D, device="cuda", dtype=torch.bfloat16)
        return s
    dtype = DTYPES[c["dtype"]]
    if c["op"] == "append":
        _cache(c, s, host, dev, dtype)
        n = s["total"]
        first = torch.repeat_interleave(s["lens"] - s["cu"].diff(), s["cu"].diff())
        local = torch.arange(n - c["pad"], device="cuda") - torch.repeat_interleave(
            s["cu"][:-1], s["cu"].diff())
        s["positions"] = torch.cat([first + local, torch.zeros(c["pad"], device="cuda")]).int()
        npos = s["kmax"]
    else:
        n = c["tokens"]
        if c["seq_len"]:
            s["positions"] = torch.arange(n, device="cuda", dtype=torch.int32) % c["seq_len"]
            npos = c["seq_len"]
        else:  # a packed batch: positions of any order, some far into a context
            npos = 32768
            s["positions"] = torch.randint(0, npos, (n,), generator=dev, device="cuda",
                                           dtype=torch.int32)
    s["table_cs"] = _rope_table(npos, c["rot"])
    # one fused projection's rows: q heads, probe heads, k heads, v heads
    heads = [Hq, Hq if c["probe"] else 0, Hkv, Hkv]
    x = (torch.randn(n, sum(heads), D, generator=dev, device="cuda") * 1.5).to(dtype)
    s["q"], r, s["k"], s["v"] = x.split(heads, 1)
    s["r"] = r if c["probe"] else None
    wt = lambda: (1 + 0.2 * torch.randn(D, generator=dev, device="cuda")).to(dtype)
    s["qw"], s["kw"] = wt(), wt()
    s["rw"] = wt() if c["probe"] and c["r_norm"] else None
    if c["op"] == "append":
        s["q_out"] = torch.zeros(n, Hq, D, device="cuda", dtype=dtype)
        s["r_out"] = torch.zeros(n, Hq, D, device="cuda", dtype=dtype) if c["probe"] else None
    if c["op"] == "rope_bwd":
        grad = lambda H: torch.randn(_out_shape(c, H), generator=dev, device="cuda").to(dtype)
        s["dq"], s["dk"] = grad(Hq), grad(Hkv)
        s["dr"] = grad(Hq) if c["probe"] else None
    return s


def _out_shape(c, H):
    n, L = c["tokens"], c["seq_len"]
    return (n // L, H, L, c["D"]) if L else (n, H, c["D"])


# ------------------------------------------------------------ plain forms ----
def _rotate(y, cs, interleaved, sign=1.0):
    """Rotate the first cs.shape[1] dimensions of y [n, H, D] by the angles of
    cs [n, rot] (backwards with sign = -1)."""
    h = cs.shape[1] // 2
    cos, sin = cs[:, None, :h], sign * cs[:, None, h:]
    a, b = (y[..., 0:2 * h:2], y[..., 1:2 * h:2]) if interleaved else (y[..., :h], y[..., h:2 * h])
    u, w = a * cos - b * sin, a * sin + b * cos
    out = y.clone()
    if interleaved:
        out[..., 0:2 * h:2], out[..., 1:2 * h:2] = u, w
    else:
        out[..., :h], out[..., h:2 * h] = u, w
    return out


def _norm_rotate(x, w, cs, interleaved):
    y = x.float()
    if w is not None:
        y = y * (1.0 / (y.square().mean(-1, keepdim=True) + EPS).sqrt()) * w.float()
    return _rotate(y, cs, interleaved)


def _norm_rotate_grad(dy, x, w, cs, interleaved):
    """(dx, dw) of _norm_rotate for the gradient dy of its output."""
    dz = _rotate(dy.float(), cs, interleaved, -1.0)
    if w is None:
        return dz, None
    xf = x.float()
    rstd = 1.0 / (xf.square().mean(-1, keepdim=True) + EPS).sqrt()
    xh = xf * rstd
    dn = dz * w.float()
    dw = (dz * xh).double().sum((0, 1)).float()
    return rstd * (dn - xh * (dn * xh).mean(-1, keepdim=True)), dw


def _to_layout(y, c):
    L = c["seq_len"]
    return y.unflatten(0, (-1, L)).transpose(1, 2).contiguous() if L else y


def _from_layout(y, c):
    return y.transpose(1, 2).flatten(0, 1) if c["seq_len"] else y


def _plain_rope(s):
    c = s["c"]
    cs = s["table_cs"][s["positions"].long()]
    f = lambda x, w: None if x is None else _to_layout(
        _norm_rotate(x, w, cs, c["interleaved"]).to(x.dtype), c)
    return f(s["q"], s["qw"]), f(s["r"], s["rw"]), f(s["k"], s["kw"])


def _plain_rope_bwd(s):
    c = s["c"]
    cs = s["table_cs"][s["positions"].long()]

    def f(dy, x, w):
        if x is None:
            return None, None
        dx, dw = _norm_rotate_grad(_from_layout(dy, c), x, w, cs, c["interleaved"])
        return dx.to(x.dtype), dw

    (dq, dqw), (dr, drw), (dk, dkw) = (f(s["dq"], s["q"], s["qw"]), f(s["dr"], s["r"], s["rw"]),
                                       f(s["dk"], s["k"], s["kw"]))
    return dq, dr, dk, dqw, drw, dkw


def _rows(s):
    """For each real token row: its sequence, and its place in that chunk."""
    cu = s["cu"].long()
    n = s["total"] - s["c"]["pad"]
    row = torch.arange(n, device="cuda")
    seq = torch.searchsorted(cu, row, right=True) - 1
    return row, seq, row - cu[seq]


def _plain_append(s):
    c = s["c"]
    row, seq, local = _rows(s)
    n = row.numel()
    cs = s["table_cs"][s["positions"].long()[:n]]
    dtype = s["q"].dtype
    s["q_out"][:n] = _norm_rotate(s["q"][:n], s["qw"], cs, c["interleaved"]).to(dtype)
    if s["r"] is not None:
        s["r_out"][:n] = _norm_rotate(s["r"][:n], s["rw"], cs, c["interleaved"]).to(dtype)
    at = s["lens"].long()[seq] - s["cu"].diff().long()[seq] + local
    page, slot = s["table"].long()[seq, at // c["page"]], at % c["page"]
    s["k_pages"][page, slot] = _norm_rotate(s["k"][:n], s["kw"], cs, c["interleaved"]).to(dtype)
    s["v_pages"][page, slot] = s["v"][:n]
    return s["q_out"], s["r_out"], s["k_pages"], s["v_pages"]


def _plain_chunk(s):
    c = s["c"]
    B, Hq, Hkv, D, G = c["B"], c["Hq"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    row, seq, local = _rows(s)
    Q, K = s["qmax"], s["kmax"]
    qlen, n = s["cu"].diff().long(), s["lens"].long()
    key = torch.arange(K, device="cuda")
    held = key < n[:, None]  # [B, K]
    page = s["table"].long()[:, key // c["page"]]
    gather = lambda pool: torch.where(held[:, :, None, None], pool[page, key % c["page"]].float(),
                                      0.0).transpose(1, 2)  # [B, Hkv, K, D]
    k, v = gather(s["k_pages"]), gather(s["v_pages"])

    def heads(x):  # the packed rows as [B, Hkv, G * Q, D]
        p = torch.zeros(B, Q, Hq, D, device="cuda")
        p[seq, local] = x[:row.numel()].float()
        return p.view(B, Q, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Q, D)

    last = (n - qlen)[:, None] + torch.arange(Q, device="cuda") if c["causal"] else (
        n[:, None] - 1).expand(B, Q)  # the last key each row sees
    seen = (held[:, None, :] & (key <= last[:, :, None]))[:, None, None]  # [B,1,1,Q,K]
    t = (heads(s["q"]) @ k.transpose(-1, -2)).mul_(D ** -0.5)
    t = t.view(B, Hkv, G, Q, K).masked_fill_(~seen, float("-inf"))
    m = t.amax(-1, keepdim=True)
    e = t.sub_(torch.where(m == float("-inf"), 0.0, m)).exp_()
    w = e.div_(e.sum(-1, keepdim=True).clamp_min(1e-30))
    if s["r"] is not None:
        p = (heads(s["r"]) @ k.transpose(-1, -2)).view(B, Hkv, G, Q, K)
        mean = (w * p).sum(-1, keepdim=True)
        w = w.mul_(p.sub_(mean).add_(1.0))
    o = w.view(B, Hkv, G * Q, K) @ v
    o = o.view(B, Hkv, G, Q, D).permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D)
    s["out"][:row.numel()] = o[seq, local].to(s["out"].dtype)
    return s["out"]


# ------------------------------------------------------- framework's calls ----
def _own(s):
    from parameterized_local_linear_b200 import binding as pl
    c = s["c"]
    op = c["op"]
    if op == "rope":
        return pl.parallax_qk_norm_rope(
            s["q"], s["r"], s["k"], s["table_cs"], s["positions"], q_weight=s["qw"],
            r_weight=s["rw"], k_weight=s["kw"], eps=EPS, interleaved=c["interleaved"],
            seq_len=c["seq_len"], workspace=_workspace(s, pl.status_workspace))
    if op == "rope_bwd":
        return pl.parallax_qk_norm_rope_backward(
            s["dq"], s["dr"], s["dk"], s["q"], s["r"], s["k"], s["table_cs"], s["positions"],
            q_weight=s["qw"], r_weight=s["rw"], k_weight=s["kw"], eps=EPS,
            interleaved=c["interleaved"], seq_len=c["seq_len"],
            workspace=_workspace(s, lambda dev: pl.norm_rope_backward_workspace(
                c["tokens"], c["Hq"], c["Hkv"], c["D"], dev)))
    if op == "append":
        pl.parallax_norm_rope_append(
            s["q"], s["r"], s["k"], s["v"], s["table_cs"], s["k_pages"], s["v_pages"], s["table"],
            s["lens"], None if c["qmax"] == 1 and not c["pad"] else s["cu"],
            positions=s["positions"], q_weight=s["qw"], r_weight=s["rw"], k_weight=s["kw"],
            eps=EPS, interleaved=c["interleaved"], q_out=s["q_out"], r_out=s["r_out"],
            workspace=_workspace(s, pl.status_workspace))
        return s["q_out"], s["r_out"], s["k_pages"], s["v_pages"]
    return pl.parallax_prefill_paged(
        s["q"], s["r"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
        None if s["qmax"] == 1 and not c["pad"] else s["cu"],
        causal=c["causal"], probe=c["probe"], out=s["out"],
        workspace=_workspace(s, lambda dev: pl.prefill_paged_workspace(
            c["B"], s["total"], c["Hq"], c["Hkv"], c["D"], dev)))


def _workspace(s, make):
    if "workspace" not in s:  # kept with the state, as a serving loop keeps it
        s["workspace"] = make(s["q"].device)
    return s["workspace"]


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "rope_bwd": _plain_rope_bwd, "append": _plain_append,
            "chunk": _plain_chunk}[state["c"]["op"]](state)


# -------------------------------------------------------------- work, exact --
def work(case):
    c = case
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    if c["op"] == "chunk":
        # K and V of every cached key once, the packed q, r and out rows, and
        # 2 D flops for each of q.k, r.k, e v, e s v of a visible pair
        qs, ns = _lengths(c)
        kv = sum(ns) * Hkv * D * 2 * 2
        rows = sum(qs) * Hq * D * (4 + 2 * c["probe"])
        pairs = sum(q * n - (q * (q - 1) / 2 if c["causal"] else 0) for q, n in zip(qs, ns))
        return {"bytes": kv + rows, "flops": pairs * Hq * D * (8 if c["probe"] else 4)}
    size = 2 if c["dtype"] == "bf16" else 4
    heads = Hq * (2 if c["probe"] else 1) + Hkv
    if c["op"] == "append":
        n = sum(_lengths(c)[0])
        return {"bytes": n * ((heads + Hkv) * 2 * D * size + c["rot"] * 4 + 4),
                "flops": n * heads * D * 7}
    n = c["tokens"]
    table = min(n, c["seq_len"] or 32768) * c["rot"] * 4
    if c["op"] == "rope":
        return {"bytes": n * (heads * 2 * D * size + 4) + table, "flops": n * heads * D * 7}
    return {"bytes": n * (heads * 3 * D * size + 4) + table, "flops": n * heads * D * 14}


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "chunk":
        return _exact_chunk(s)
    D = c["D"]
    n = s["q"].shape[0] - c.get("pad", 0)
    cs = s["table_cs"].double()[s["positions"][:n].long()]
    half = c["rot"] // 2
    # pair p of a head: dimensions (2 p, 2 p + 1), or (p, p + half)
    p = torch.arange(half, device="cuda")
    ia, ib = (2 * p, 2 * p + 1) if c["interleaved"] else (p, p + half)
    # the rotation of each token as a D x D matrix
    R = torch.eye(D, device="cuda", dtype=torch.float64).repeat(min(n, 256), 1, 1)

    def blocks(x):
        for a in range(0, n, 256):
            m = min(256, n - a)
            M = R[:m].clone()
            co, si = cs[a:a + m, :half], cs[a:a + m, half:]
            M[:, ia, ia], M[:, ib, ib] = co, co
            M[:, ia, ib], M[:, ib, ia] = -si, si
            yield slice(a, a + m), M

    def forward(x, w):
        if x is None:
            return None
        out = torch.empty(n, x.shape[1], D, device="cuda", dtype=torch.float64)
        for at, M in blocks(x):
            y = x[at].double()
            if w is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + EPS) * w.double()
            out[at] = torch.einsum("nij,nhj->nhi", M, y)
        return out

    def backward(dy, x, w):
        if x is None:
            return None, None
        dx = torch.empty(n, x.shape[1], D, device="cuda", dtype=torch.float64)
        dw = torch.zeros(D, device="cuda", dtype=torch.float64)
        for at, M in blocks(x):
            dz = torch.einsum("nij,nhi->nhj", M, dy[at].double())
            if w is None:
                dx[at] = dz
                continue
            y = x[at].double()
            v = (y * y).sum(-1, keepdim=True) / D + EPS
            dw += torch.einsum("nhj,nhj->j", dz, y / torch.sqrt(v))
            dn = dz * w.double()
            dx[at] = dn / torch.sqrt(v) - y * (dn * y).sum(-1, keepdim=True) / (D * v * torch.sqrt(v))
        return dx, None if w is None else dw

    if c["op"] == "rope":
        got = forward(s["q"], s["qw"]), forward(s["r"], s["rw"]), forward(s["k"], s["kw"])
        return tuple(None if y is None else _to_layout(y, c) for y in got)
    if c["op"] == "rope_bwd":
        f = lambda d, x, w: backward(None if x is None else _from_layout(d, c), x, w)
        (dq, dqw), (dr, drw), (dk, dkw) = (f(s["dq"], s["q"], s["qw"]),
                                           f(s["dr"], s["r"], s["rw"]),
                                           f(s["dk"], s["k"], s["kw"]))
        return dq, dr, dk, dqw, drw, dkw
    q, r, k = (forward(None if x is None else x[:n], w) for x, w in (
        (s["q"], s["qw"]), (s["r"], s["rw"]), (s["k"], s["kw"])))
    pad = lambda y: None if y is None else torch.cat(
        [y, torch.zeros(c["pad"], *y.shape[1:], device="cuda", dtype=torch.float64)])
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    at = 0
    for b in range(c["B"]):
        for j in range(s["qs"][b]):
            i = s["ns"][b] - s["qs"][b] + j
            page, slot = divmod(i, c["page"])
            page = int(s["table"][b, page]) if j == 0 or slot == 0 else held
            held = page
            kp[page, slot], vp[page, slot] = k[at], s["v"][at].double()
            at += 1
    return pad(q), pad(r), kp, vp


def _exact_chunk(s):
    c = s["c"]
    G, D, ps = c["Hq"] // c["Hkv"], c["D"], c["page"]
    out = torch.zeros(s["total"], c["Hq"], D, device="cuda", dtype=torch.float64)
    table = s["table"].cpu()
    at = 0
    for b in range(c["B"]):
        nq, n = s["qs"][b], s["ns"][b]
        pages = table[b, :-(-n // ps)].long().cuda()
        key = torch.arange(n, device="cuda")
        for g in range(c["Hkv"]):
            k = s["k_pages"][pages, :, g].reshape(-1, D)[:n].double()
            v = s["v_pages"][pages, :, g].reshape(-1, D)[:n].double()
            for h in range(g * G, g * G + G):
                for j0 in range(0, nq, 1024):
                    j1 = min(nq, j0 + 1024)
                    rows = slice(at + j0, at + j1)
                    pos = torch.arange(n - nq + j0, n - nq + j1, device="cuda")
                    t = s["q"][rows, h].double() @ k.T / math.sqrt(D)
                    if c["causal"]:
                        t = t.masked_fill(key > pos[:, None], float("-inf"))
                    w = torch.softmax(t, -1)
                    o = w @ v
                    if s["r"] is not None:
                        # sum_i w_i (s_i - sbar)(v_i - vbar)
                        sc = s["r"][rows, h].double() @ k.T
                        w = w * (sc - (w * sc).sum(-1, keepdim=True))
                        o = o + w @ v - w.sum(-1, keepdim=True) * o
                    out[rows, h] = o
        at += nq
    return out
