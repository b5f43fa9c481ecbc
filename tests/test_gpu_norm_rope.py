"""GPU tests of the norm and rotation of the heads (parallax_qk_norm_rope, its
backward pass and parallax_norm_rope_append) against the formulas in 64 bits.

Tolerances count roundings (u = 2^-24 of fp32, half a step of the output type):
a value n = x rstd w carries at most 20 u (the sum of squares of 128 values in 16
serial and 3 or 2 tree steps, its root and reciprocal, two products), and the
rotation adds two products and a sum: 24 u of |n_a| + |n_b| in all. A row gradient
is rstd (dn - xh mean(dn xh)) with two such sums: 48 u of rstd (|dn| + |xh|
mean|dn xh|). A weight gradient adds at most 60 terms one after the other at
these sizes (a lane's rows, the lanes, warps and blocks), each within 30 u:
90 u of sum |dz xh|."""
import pytest
import torch

from parameterized_local_linear_b200 import binding as pl

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
EPS = 1e-6


def rotate(y, cs, interleaved, sign=1.0):
    h = cs.shape[1] // 2
    cos, sin = cs[:, None, :h], sign * cs[:, None, h:]
    ia = torch.arange(h, device=y.device) * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else h)
    out = y.clone()
    out[..., ia] = y[..., ia] * cos - y[..., ib] * sin
    out[..., ib] = y[..., ia] * sin + y[..., ib] * cos
    return out


def spread(y, rot, interleaved):
    """|y_a| + |y_b| of each dimension's pair (|y| past rot)."""
    h = rot // 2
    ia = torch.arange(h, device=y.device) * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else h)
    out = y.abs().clone()
    out[..., ia] = out[..., ib] = y[..., ia].abs() + y[..., ib].abs()
    return out


def normed(x, w):
    x = x.double()
    return x if w is None else x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w.double()


def check(got, want, slack, dtype, what):
    err = (got.double() - want).abs()
    tol = HALF[dtype] * want.abs() + slack
    assert got.dtype == dtype and got.shape == want.shape
    bad = ~(err <= tol)
    assert not bad.any(), (what, err[bad].max().item(), (err / tol.clamp_min(1e-300)).max().item())


def layout(y, L):
    return y.unflatten(0, (-1, L)).transpose(1, 2).contiguous() if L else y


def inputs(n, Hq, Hkv, D, rot, dtype, seed, npos=4096, fused=True, r=True, v=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    heads = [Hq, Hq, Hkv, Hkv]
    x = (torch.randn(n, sum(heads), D, device="cuda", generator=g) * 2).to(dtype)
    parts = list(x.split(heads, 1)) if fused else [p.contiguous() for p in x.split(heads, 1)]
    w = [(1 + 0.3 * torch.randn(D, device="cuda", generator=g)).to(dtype) for _ in range(3)]
    pos = torch.randint(0, npos, (n,), device="cuda", generator=g, dtype=torch.int32)
    cs = pl.parallax_rope_table(npos, rot, 1e4)
    return (parts if r else [parts[0], None, *parts[2:]]), w, pos, cs


@pytest.mark.parametrize("rot", [16, 64, 96, 128])
def test_table(rot):
    cs = pl.parallax_rope_table(70000, rot, 1e6)
    t = torch.arange(70000, dtype=torch.float64, device="cuda")[:, None]
    ang = t * 1e6 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    want = torch.cat([ang.cos(), ang.sin()], 1)
    # the angle in fp64: 70000 x 2^-53 times a few steps, then half a step of fp32
    assert ((cs.double() - want).abs() <= U * want.abs() + 1e-10).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 96), (128, 16), (64, 64), (64, 32)])
@pytest.mark.parametrize("n,Hq,Hkv", [(1, 1, 1), (7, 6, 2), (50, 16, 8), (500, 16, 8)])
def test_forward(n, Hq, Hkv, D, rot, interleaved, dtype):
    (q, r, k, _), w, pos, cs = inputs(n, Hq, Hkv, D, rot, dtype, seed=n + rot)
    for weights, probe in ((w, True), ([w[0], None, w[2]], True), ([None] * 3, False)):
        got = pl.parallax_qk_norm_rope(q, r if probe else None, k, cs, pos, *weights,
                                       interleaved=interleaved)
        assert (got[1] is None) == (not probe)
        for x, wt, o in zip((q, r, k), weights, got):
            if o is None:
                continue
            y = normed(x, wt)
            check(o, rotate(y, cs[pos.long()].double(), interleaved),
                  24 * U * spread(y, rot, interleaved), dtype, (n, D, rot, wt is None))


@pytest.mark.parametrize("L", [1, 5, 40])
def test_batched_layout_and_default_positions(L):
    n, Hq, Hkv, D = 3 * L, 4, 2, 128
    (q, r, k, _), w, _, cs = inputs(n, Hq, Hkv, D, 128, torch.bfloat16, seed=L)
    pos = torch.arange(n, device="cuda", dtype=torch.int32) % L
    flat = pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w)
    got = pl.parallax_qk_norm_rope(q, r, k, cs, None, *w, seq_len=L)
    for a, b in zip(flat, got):
        assert torch.equal(layout(a, L), b)
    # packed without positions: 0, 1, ...
    a = pl.parallax_qk_norm_rope(q, r, k, cs, None, *w)
    b = pl.parallax_qk_norm_rope(q, r, k, cs, torch.arange(n, device="cuda", dtype=torch.int32), *w)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_in_place_and_given_outputs():
    (q, r, k, _), w, pos, cs = inputs(65, 4, 2, 64, 64, torch.bfloat16, seed=3, fused=False)
    want = pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w)
    out = pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w, out=(q, r, k))
    assert out[0].data_ptr() == q.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(want, (q, r, k)))


def test_nonfinite_values_stay_in_their_row():
    (q, r, k, _), w, pos, cs = inputs(9, 4, 2, 128, 64, torch.bfloat16, seed=4)
    want = pl.parallax_qk_norm_rope(q, r, k, cs, pos, w[0], None, w[2])
    q[3, 1, 5] = float("nan")
    r[2, 2, 100] = float("inf")  # no norm, past the rotated dimensions
    got = pl.parallax_qk_norm_rope(q, r, k, cs, pos, w[0], None, w[2])
    assert got[0][3, 1].isnan().all()
    got[0][3, 1] = want[0][3, 1]
    assert got[1][2, 2, 100] == float("inf")
    got[1][2, 2, 100] = want[1][2, 2, 100]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_past_32_bit_offsets():
    """More than 2^31 elements of q: the last tokens are those of a small call, in
    the packed and in the batched layout, forward and backward."""
    n, Hq, Hkv, D = 1_050_000, 16, 1, 128
    assert n * Hq * D > 2 ** 31
    q = torch.zeros(n, Hq, D, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(n, Hkv, D, device="cuda", dtype=torch.bfloat16)
    m = 50
    (sq, _, sk, _), w, _, cs = inputs(m, Hq, Hkv, D, D, torch.bfloat16, seed=70)
    q[-m:], k[-m:] = sq, sk
    pos = torch.zeros(n, device="cuda", dtype=torch.int32)
    pos[-m:] = torch.arange(m, device="cuda", dtype=torch.int32)
    args = (w[0], None, w[2])
    want = pl.parallax_qk_norm_rope(sq, None, sk, cs, pos[-m:], *args)
    got = pl.parallax_qk_norm_rope(q, None, k, cs, pos, *args)
    assert torch.equal(got[0][-m:], want[0]) and torch.equal(got[2][-m:], want[2])
    assert not got[0][:-m].any()
    wantg = pl.parallax_qk_norm_rope_backward(want[0], None, want[2], sq, None, sk, cs, pos[-m:], *args)
    gotg = pl.parallax_qk_norm_rope_backward(*got, q, None, k, cs, pos, *args)
    assert torch.equal(gotg[0][-m:], wantg[0]) and torch.equal(gotg[2][-m:], wantg[2])
    del got, gotg
    L = n // 2
    y = pl.parallax_qk_norm_rope(q, None, k, cs, pos, *args, seq_len=L)
    assert torch.equal(y[0][1, :, -m:].transpose(0, 1), want[0])
    assert torch.equal(y[2][1, :, -m:].transpose(0, 1), want[2])


def test_zero_rows_and_position_clamp():
    (q, r, k, _), w, pos, cs = inputs(6, 4, 2, 64, 64, torch.float32, seed=5, npos=100)
    q.zero_()
    pos[:3] = torch.tensor([-1, 100, 2 ** 31 - 1])
    ws = pl.status_workspace("cuda")
    got = pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w, workspace=ws)
    assert (got[0] == 0).all()
    fixed = pos.clamp(0, 99)
    want = pl.parallax_qk_norm_rope(q, r, k, cs, fixed, *w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert int(ws[:4].view(torch.int32)) == 4


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 32), (64, 64), (64, 48)])
@pytest.mark.parametrize("n,Hq,Hkv", [(1, 1, 1), (7, 6, 2), (130, 16, 8)])
def test_backward(n, Hq, Hkv, D, rot, interleaved, dtype):
    (q, r, k, _), w, pos, cs = inputs(n, Hq, Hkv, D, rot, dtype, seed=n + rot + 1)
    g = torch.Generator(device="cuda").manual_seed(9)
    dy = [torch.randn(n, H, D, device="cuda", generator=g).to(dtype) for H in (Hq, Hq, Hkv)]
    c64 = cs[pos.long()].double()
    for weights, probe in ((w, True), ([w[0], None, w[2]], True), ([None] * 3, False)):
        got = pl.parallax_qk_norm_rope_backward(dy[0], dy[1] if probe else None, dy[2], q,
                                                r if probe else None, k, cs, pos, *weights,
                                                interleaved=interleaved)
        for i, (x, wt, d) in enumerate(zip((q, r, k), weights, dy)):
            if i == 1 and not probe:
                assert got[1] is None and got[4] is None
                continue
            dz = rotate(d.double(), c64, interleaved, -1.0)
            sz = spread(d.double(), rot, interleaved)
            if wt is None:
                check(got[i], dz, 4 * U * sz, dtype, "dx")
                assert got[3 + i] is None
                continue
            xd = x.double()
            rstd = 1 / torch.sqrt(xd.square().mean(-1, keepdim=True) + EPS)
            xh, dn, sn = xd * rstd, dz * wt.double(), sz * wt.double().abs()
            dx = rstd * (dn - xh * (dn * xh).mean(-1, keepdim=True))
            check(got[i], dx, 48 * U * rstd * (sn + xh.abs() * (sn * xh.abs()).mean(-1, keepdim=True)),
                  dtype, "dx")
            check(got[3 + i], (dz * xh).sum((0, 1)), 90 * U * (sz * xh.abs()).sum((0, 1)),
                  torch.float32, "dw")


def test_backward_against_differences():
    """Central differences of the fp64 formula along random directions, and the
    same of the kernel's own forward (fp32, a large step)."""
    n, Hq, Hkv, D, rot = 5, 4, 2, 64, 32
    (q, r, k, _), w, pos, cs = inputs(n, Hq, Hkv, D, rot, torch.float32, seed=21)
    g = torch.Generator(device="cuda").manual_seed(22)
    dy = [torch.randn(n, H, D, device="cuda", generator=g) for H in (Hq, Hq, Hkv)]
    got = pl.parallax_qk_norm_rope_backward(*dy, q, r, k, cs, pos, *w)
    c64 = cs[pos.long()].double()
    for i, (x, wt) in enumerate(zip((q, r, k), w)):
        dirx = torch.randn(x.shape, device="cuda", generator=g).double()
        dirw = torch.randn(D, device="cuda", generator=g).double()
        f = lambda h: (rotate(normed(x.double() + h * dirx, wt.double() + h * dirw), c64, False)
                       * dy[i].double()).sum()
        h = 1e-5
        want = (f(h) - f(-h)) / (2 * h)
        have = (got[i].double() * dirx).sum() + (got[3 + i].double() * dirw).sum()
        # 500 terms of order 1, each within 1e-6 of its own; the difference formula
        # is off by h^2 times the third derivative and 2^-53 / h times the value
        assert abs(have - want) <= 2e-4 * max(1.0, abs(want)), (i, have, want)


def test_backward_layouts_strided_gradients_and_repeat():
    n, L, Hq, Hkv, D = 60, 20, 4, 2, 128
    (q, r, k, _), w, _, cs = inputs(n, Hq, Hkv, D, 128, torch.bfloat16, seed=30)
    g = torch.Generator(device="cuda").manual_seed(31)
    dy = [torch.randn(n, H, D, device="cuda", generator=g).bfloat16() for H in (Hq, Hq, Hkv)]
    pos = torch.arange(n, device="cuda", dtype=torch.int32) % L
    flat = pl.parallax_qk_norm_rope_backward(*dy, q, r, k, cs, pos, *w)
    whole = torch.full((n, 2 * Hq + 2 * Hkv, D), 7.0, device="cuda", dtype=torch.bfloat16)
    out = whole.split([Hq, Hq, Hkv, Hkv], 1)
    got = pl.parallax_qk_norm_rope_backward(*(layout(d, L) for d in dy), q, r, k, cs, None, *w,
                                            seq_len=L, out=out[:3])
    for a, b in zip(flat, got):
        assert torch.equal(a, b)
    assert (out[3] == 7).all()  # the value heads' slice is not touched
    again = pl.parallax_qk_norm_rope_backward(*dy, q, r, k, cs, pos, *w)
    assert all(torch.equal(a, b) for a, b in zip(flat, again))
    # in place of the incoming gradients
    d = [x.clone() for x in dy]
    pl.parallax_qk_norm_rope_backward(*d, q, r, k, cs, pos, *w, out=d)
    assert all(torch.equal(a, b) for a, b in zip(flat, d))


# ------------------------------------------------------------------ append --
def make_cache(seqs, ps, Hkv, D, dtype, seed, extra=2):
    """Pools, a table of distinct pages in random order, cu and lens."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(n, 1) // ps) for _, n in seqs]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=g).int()
    table = torch.full((len(seqs), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    pool = lambda s: torch.randn(pages, ps, Hkv, D, generator=torch.Generator().manual_seed(s)).to(dtype)
    cu = torch.zeros(len(seqs) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor([q for q, _ in seqs]).cumsum(0)
    lens = torch.tensor([n for _, n in seqs], dtype=torch.int32)
    return [x.cuda() for x in (pool(seed), pool(seed + 1), table, cu, lens)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 16, 8), (64, 3, 1)])
@pytest.mark.parametrize("seqs,ps,pad", [
    ([(1, 1)], 64, 0), ([(1, 64), (1, 65), (1, 300)], 64, 0),
    ([(5, 5), (0, 70), (130, 200), (0, 0), (1, 129)], 64, 9),
    ([(3, 10)] * 70, 16, 1)])
def test_append(seqs, ps, pad, D, Hq, Hkv, dtype):
    kp, vp, table, cu, lens = make_cache(seqs, ps, Hkv, D, dtype, seed=40)
    n = int(cu[-1]) + pad
    (q, r, k, v), w, _, cs = inputs(n, Hq, Hkv, D, D, dtype, seed=41)
    want_kp, want_vp = kp.clone(), vp.clone()
    idx = torch.cat([torch.arange(nn - c, nn) for c, nn in seqs]).cuda()
    idx = torch.cat([idx, torch.zeros(pad, device="cuda", dtype=idx.dtype)]).int()
    fq, fr, fk = pl.parallax_qk_norm_rope(q, r, k, cs, idx, *w)  # tested above
    seq = torch.repeat_interleave(torch.arange(len(seqs)), torch.tensor([c for c, _ in seqs])).cuda()
    m = n - pad
    page = table.long()[seq, idx[:m].long() // ps]
    want_kp[page, idx[:m].long() % ps] = fk[:m]
    want_vp[page, idx[:m].long() % ps] = v[:m]
    qo = torch.full((n, Hq, D), 3.0, device="cuda", dtype=dtype)
    ro = qo.clone()
    ws = pl.status_workspace("cuda")
    pl.parallax_norm_rope_append(q, r, k, v, cs, kp, vp, table, lens, cu, None, *w, q_out=qo,
                                 r_out=ro, workspace=ws)
    assert torch.equal(kp, want_kp) and torch.equal(vp, want_vp)
    assert torch.equal(qo[:m], fq[:m]) and torch.equal(ro[:m], fr[:m])
    assert (qo[m:] == 3).all() and (ro[m:] == 3).all()  # rows past the last sequence
    assert int(ws[:4].view(torch.int32)) == 0
    if all(c == 1 for c, _ in seqs):  # one token per sequence: no cu_seqlens needed
        kp2, vp2, *_ = make_cache(seqs, ps, Hkv, D, dtype, seed=40)
        q2, r2 = pl.parallax_norm_rope_append(q, r, k, v, cs, kp2, vp2, table, lens, None, None, *w)
        assert torch.equal(q2, fq) and torch.equal(kp2, want_kp) and torch.equal(vp2, want_vp)


def test_append_positions_without_probe_and_bad_slots():
    seqs, ps, Hq, Hkv, D = [(4, 70), (3, 3), (2, 66)], 64, 4, 2, 64
    kp, vp, table, cu, lens = make_cache(seqs, ps, Hkv, D, torch.bfloat16, seed=50)
    (q, _, k, v), w, pos, cs = inputs(9, Hq, Hkv, D, 32, torch.bfloat16, seed=51)
    want = pl.parallax_qk_norm_rope(q, None, k, cs, pos, w[0], None, w[2], interleaved=True)
    base_k, base_v = kp.clone(), vp.clone()
    ws = pl.status_workspace("cuda")
    run = lambda t, n: pl.parallax_norm_rope_append(q, None, k, v, cs, kp, vp, t, n, cu, pos, w[0],
                                                    None, w[2], interleaved=True, workspace=ws)
    qo, ro = run(table, lens)
    assert ro is None and torch.equal(qo, want[0]) and int(ws[:4].view(torch.int32)) == 0
    assert torch.equal(kp[table[0, 1], 2:6], want[2][:4]) and torch.equal(vp[table[1, 0], :3], v[4:7])
    # a page outside the pool, a length that puts keys before 0, one past the table:
    # those keys are not written, everything else is
    for t, n in ((table.clone(), lens.clone()), (table, lens.clone()), (table, lens.clone())):
        kp.copy_(base_k), vp.copy_(base_v), ws.zero_()
        want_k, want_v = base_k.clone(), base_v.clone()
        if t is not table:
            t[2, 1] = kp.shape[0]
            keep = [(0, range(4)), (1, range(3))]
        elif keep is not None and len(keep) == 2:
            n[1] = 1  # tokens 4, 5 before the first key
            keep = [(0, range(4)), (1, range(2, 3)), (2, range(2))]
        else:
            n[0] = 2 ** 31 - 1
            keep = [(1, range(3)), (2, range(2))]
        for b, js in keep:
            for j in js:
                i = int(n[b]) - seqs[b][0] + j
                want_k[t[b, i // ps], i % ps] = want[2][int(cu[b]) + j]
                want_v[t[b, i // ps], i % ps] = v[int(cu[b]) + j]
        qo, _ = run(t, n)
        assert torch.equal(kp, want_k) and torch.equal(vp, want_v) and torch.equal(qo, want[0])
        assert int(ws[:4].view(torch.int32)) == 2


def test_append_idle_rows_in_place_and_default_positions():
    """One token per sequence, two of them idle (length 0): no output, no slot,
    no status. q and r are their own outputs."""
    Hq, Hkv, D, ps = 8, 2, 128, 16
    seqs = [(1, 5), (1, 0), (1, 33), (1, 0), (1, 16)]
    kp, vp, table, _, lens = make_cache(seqs, ps, Hkv, D, torch.bfloat16, seed=52)
    (q, r, k, v), w, _, cs = inputs(5, Hq, Hkv, D, D, torch.bfloat16, seed=53, fused=False)
    live = torch.tensor([0, 2, 4], device="cuda")
    pos = (lens - 1).clamp(min=0)
    fq, fr, fk = pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w)
    want_q, want_r, want_k, want_v = q.clone(), r.clone(), kp.clone(), vp.clone()
    want_q[live], want_r[live] = fq[live], fr[live]
    for b in live.tolist():
        page, at = int(table[b, int(pos[b]) // ps]), int(pos[b]) % ps
        want_k[page, at], want_v[page, at] = fk[b], v[b]
    ws = pl.status_workspace("cuda")
    qo, ro = pl.parallax_norm_rope_append(q, r, k, v, cs, kp, vp, table, lens, None, None, *w,
                                          q_out=q, r_out=r, workspace=ws)
    assert qo.data_ptr() == q.data_ptr()
    for got, want in ((q, want_q), (r, want_r), (kp, want_k), (vp, want_v)):
        assert torch.equal(got, want)
    assert int(ws[:4].view(torch.int32)) == 0


def test_backward_calls_sharing_a_workspace():
    """Calls of other sizes, head sizes and weights one after the other on one
    workspace: the block counters are 0 again after each."""
    sizes = [(1, 1, 1, 64), (700, 16, 8, 128), (3, 6, 2, 64), (700, 16, 8, 128), (90, 16, 16, 128)]
    nbytes = max(pl.norm_rope_backward_workspace(*s, "cuda").numel() for s in sizes)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
    for j, (n, Hq, Hkv, D) in enumerate(sizes):
        (q, r, k, _), w, pos, cs = inputs(n, Hq, Hkv, D, D, torch.float32, seed=54 + j)
        if j == 4:
            w[1] = None
        dy = [x.contiguous() for x in (r, q, k)]
        want = pl.parallax_qk_norm_rope_backward(*dy, q, r, k, cs, pos, *w)
        got = pl.parallax_qk_norm_rope_backward(*dy, q, r, k, cs, pos, *w, workspace=ws)
        for a, b in zip(want, got):
            assert (a is None and b is None) or torch.equal(a, b)
    assert not ws[:256].any()


def test_table_on_a_stream():
    want = pl.parallax_rope_table(500, 64, 1e4)
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = pl.parallax_rope_table(500, 64, 1e4, stream=stream)
        s.synchronize()
        assert torch.equal(got, want)


def test_streams_graphs_and_devices_context():
    """On another stream, and captured twice with separate workspaces."""
    (q, r, k, _), w, pos, cs = inputs(300, 8, 4, 128, 128, torch.bfloat16, seed=60)
    want = pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w)
    dy = [x.clone() for x in want]
    wantg = pl.parallax_qk_norm_rope_backward(*dy, q, r, k, cs, pos, *w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w, stream=s)
    gotg = pl.parallax_qk_norm_rope_backward(*dy, q, r, k, cs, pos, *w, stream=s.cuda_stream)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(wantg, gotg))
    graphs = []
    for _ in range(2):
        ws = pl.norm_rope_backward_workspace(300, 8, 4, 128, q.device)
        out = tuple(torch.empty_like(x) for x in want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w, out=out, workspace=ws)
            grads = pl.parallax_qk_norm_rope_backward(*dy, q, r, k, cs, pos, *w, workspace=ws)
        graphs.append((graph, out, grads, ws))
    for graph, *_ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for _, out, grads, _ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))
        assert all(torch.equal(a, b) for a, b in zip(wantg, grads))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 16, 8), (64, 6, 2)])
def test_append_made_outputs_hold_zeros_without_a_token(D, Hq, Hkv, dtype):
    """Padding rows (also in front) and idle rows of outputs that the call allocates,
    from memory that held NaN before; a given output keeps them."""
    seqs, ps, n = [(1, 5), (0, 9), (30, 33), (1, 16)], 16, 60
    kp, vp, table, cu, lens = make_cache(seqs, ps, Hkv, D, dtype, seed=120)
    (q, r, k, v), w, _, cs = inputs(n, Hq, Hkv, D, D, dtype, seed=121)

    def run(cu, lens, m, **out):
        junk = [torch.full((m, Hq, D), float("nan"), device="cuda", dtype=dtype) for _ in range(8)]
        del junk
        return pl.parallax_norm_rope_append(q[:m], r[:m], k[:m], v[:m], cs, kp, vp, table, lens, cu,
                                            None, *w, **out)

    kept = lambda m: torch.full((m, Hq, D), 3.0, device="cuda", dtype=dtype)
    one = torch.tensor([5, 0, 33, 0], dtype=torch.int32, device="cuda")
    for c, nn, m, live in ((cu + 7, lens, n, range(7, 39)), (None, one, 4, (0, 2))):
        rest = torch.ones(m, dtype=torch.bool)
        rest[list(live)] = False
        rest = rest.cuda()
        a, b = run(c, nn, m)
        given = run(c, nn, m, q_out=kept(m), r_out=kept(m))
        half = run(c, nn, m, q_out=kept(m)), run(c, nn, m, r_out=kept(m))
        assert not a[rest].any() and not b[rest].any()
        assert (given[0][rest] == 3).all() and (given[1][rest] == 3).all()
        assert (half[0][0][rest] == 3).all() and not half[0][1][rest].any()
        assert not half[1][0][rest].any() and (half[1][1][rest] == 3).all()
        for x in (given, *half):
            assert torch.equal(x[0][~rest], a[~rest]) and torch.equal(x[1][~rest], b[~rest])
        assert a[~rest].isfinite().all() and b[~rest].isfinite().all()


# ---------------------------------------------------------------- autograd --
def leaves(n, Hq, Hkv, D, dtype, seed):
    """One fused projection's rows and the weights, all requiring gradients."""
    (q, r, k, v), w, pos, cs = inputs(n, Hq, Hkv, D, D, dtype, seed)
    x = torch.cat([q, r, k, v], 1).requires_grad_()
    return x, [t.requires_grad_() for t in w], pos, cs, [Hq, Hq, Hkv, Hkv]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L", [0, 10])
def test_autograd_gives_the_backward_passes_gradients(L, dtype):
    """Through slices of a fused projection: x.grad is the slices' gradients, each
    weight's its own in the weight's type, and the outputs are those without autograd."""
    n, Hq, Hkv, D = 30, 4, 2, 64
    x, w, pos, cs, heads = leaves(n, Hq, Hkv, D, dtype, 130)
    pos = None if L else pos
    q, r, k, _ = x.split(heads, 1)
    out = pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w, seq_len=L)
    with torch.no_grad():
        plain = pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w, seq_len=L)
    assert all(torch.equal(a, b) and a.requires_grad and not b.requires_grad
               for a, b in zip(out, plain))
    g = torch.Generator(device="cuda").manual_seed(131)
    dy = [torch.randn(o.shape, device="cuda", generator=g).to(dtype) for o in out]
    torch.autograd.backward(out, dy)
    with torch.no_grad():
        want = pl.parallax_qk_norm_rope_backward(*dy, q, r, k, cs, pos, *w, seq_len=L)
    for a, b in zip(x.grad.split(heads, 1), want[:3]):
        assert torch.equal(a, b)
    assert not x.grad[:, -Hkv:].any()
    for t, b in zip(w, want[3:]):
        assert t.grad.dtype == dtype and torch.equal(t.grad, b.to(dtype))


def test_autograd_of_some_inputs_and_outputs():
    """Without a probe, weights that want no gradient, an output that is not used,
    and gradients that are broadcast or not aligned."""
    n, Hq, Hkv, D = 9, 4, 2, 64
    (q, r, k, _), w, pos, cs = inputs(n, Hq, Hkv, D, D, torch.float32, seed=132, fused=False)
    q.requires_grad_()
    w[2].requires_grad_()
    ones = lambda H: torch.ones(n, H, D, device="cuda")
    oq, o_r, ok = pl.parallax_qk_norm_rope(q, None, k, cs, pos, w[0], None, w[2])
    assert o_r is None
    oq.sum().backward()  # an expanded gradient; ok is not used
    with torch.no_grad():
        want = pl.parallax_qk_norm_rope_backward(ones(Hq), None, torch.zeros_like(k), q, None, k, cs,
                                                 pos, w[0], None, w[2])
    assert torch.equal(q.grad, want[0]) and not w[2].grad.any() and w[0].grad is None
    odd = torch.zeros(n * Hkv * D + 1, device="cuda")[1:].view(n, Hkv, D).copy_(ones(Hkv))
    assert odd.data_ptr() % 16
    out = pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w)
    (dk,) = torch.autograd.grad(out[2], [w[2]], odd)
    with torch.no_grad():
        want = pl.parallax_qk_norm_rope_backward(torch.zeros_like(q), torch.zeros_like(r), ones(Hkv),
                                                 q, r, k, cs, pos, *w)
    assert torch.equal(dk, want[5])
    # weights without a norm on the probe, and a stream of its own
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    r.requires_grad_()
    out = pl.parallax_qk_norm_rope(q, r, k, cs, pos, w[0], None, w[2], stream=s)
    s.synchronize()
    (dr,) = torch.autograd.grad(out[1], [r], ones(Hq))
    torch.cuda.synchronize()
    with torch.no_grad():
        want = pl.parallax_qk_norm_rope_backward(torch.zeros_like(q), ones(Hq), torch.zeros_like(k),
                                                 q, r, k, cs, pos, w[0], None, w[2])
    assert torch.equal(dr, want[1])


def test_autograd_refusals():
    (q, r, k, _), w, pos, cs = inputs(5, 4, 2, 64, 64, torch.float32, seed=133, fused=False)
    w[0].requires_grad_()
    out = tuple(torch.empty_like(x) for x in (q, r, k))
    with pytest.raises(ValueError):
        pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w, out=out)
    with pytest.raises(ValueError):
        pl.parallax_qk_norm_rope(q, r, k, cs.clone().requires_grad_(), pos, *w)
    with torch.no_grad():
        pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w, out=out)
    # once differentiable
    oq, _, _ = pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w)
    (g,) = torch.autograd.grad(oq.square().sum(), [w[0]], create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_autograd_captured_in_a_graph():
    """Forward and gradients in one graph, replayed on other inputs, while an eager
    graph of the same leaves lives on another stream. (One on the default stream
    breaks the capture of any operator's gradients: torch keeps a leaf's accumulation
    on the stream where it was first used.)"""
    n, Hq, Hkv, D = 200, 8, 4, 128
    x, w, pos, cs, heads = leaves(n, Hq, Hkv, D, torch.bfloat16, 134)
    dy = [torch.randn(n, H, D, device="cuda").bfloat16() for H in heads[:3]]

    def step():
        out = pl.parallax_qk_norm_rope(*x.split(heads, 1)[:3], cs, pos, *w)
        return out, torch.autograd.grad(out, [x, *w], dy)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        alive, _ = step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, grads = step()
    for _ in range(2):
        with torch.no_grad():
            x.copy_(x.roll(3, 0))
        graph.replay()
        want_out, want = step()
        assert all(torch.equal(a, b) for a, b in zip((*out, *grads), (*want_out, *want)))
    assert alive[0].requires_grad


def test_status_of_the_workspaces_that_calls_take():
    """parallax_workspace_status reads (and clears) the tensors that the norm, rotation
    and chunk calls take, as it does a decode's Workspace."""
    (q, r, k, _), w, pos, cs = inputs(6, 4, 2, 64, 64, torch.float32, seed=140, npos=100)
    for ws in (pl.status_workspace("cuda"), pl.norm_rope_backward_workspace(6, 4, 2, 64, "cuda"),
               pl.prefill_paged_workspace(1, 6, 4, 2, 64, "cuda"), pl.Workspace(1, 4, 2, 64, 64)):
        assert pl.parallax_workspace_status(ws) == (0, 0)
        pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w, workspace=ws)
        assert pl.parallax_workspace_status(ws) == (0, 0)
        pl.parallax_qk_norm_rope(q, r, k, cs, pos + 100, *w, workspace=ws)
        assert pl.parallax_workspace_status(ws, clear=True) == (-13, 4)
        assert pl.parallax_workspace_status(ws) == (0, 0)


@pytest.mark.parametrize("n", [1, 40, 3000])
def test_bounded_wait_reports_and_context_survives(n):
    """The first rows of each kind are never loaded: within the short limit the status
    word says so (no matter how few of the ring's stages hold copies), the rows of other
    warps are right, the backward's counters are 0 again and the next calls are right."""
    import time
    Hq, Hkv, D, ps = 16, 8, 128, 64
    (q, r, k, v), w, pos, cs = inputs(n, Hq, Hkv, D, D, torch.bfloat16, seed=141)
    dy = [torch.randn(n, H, D, device="cuda").bfloat16() for H in (Hq, Hq, Hkv)]
    kp, vp, table, cu, lens = make_cache([(n, n)], ps, Hkv, D, torch.bfloat16, seed=142)
    ws = pl.norm_rope_backward_workspace(n, Hq, Hkv, D, "cuda")
    q_out = torch.empty(n, Hq, D, device="cuda", dtype=torch.bfloat16)
    calls = (
        lambda: pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w, workspace=ws),
        lambda: pl.parallax_qk_norm_rope_backward(*dy, q, r, k, cs, pos, *w, workspace=ws),
        lambda: pl.parallax_norm_rope_append(q, r, k, v, cs, kp, vp, table, lens, cu, pos, *w,
                                             q_out=q_out, r_out=torch.empty_like(q_out), workspace=ws),
    )
    stall = pl.load_library().parallax_testing_norm_rope_stall_next
    for call in calls:
        want = [x.clone() for x in call()]
        torch.cuda.synchronize()
        start = time.perf_counter()
        assert stall(50) == 0
        got = call()
        assert pl.parallax_workspace_status(ws) == (-9, 1)
        assert 0.04 < time.perf_counter() - start < 1.5  # 50 ms for each of at most 3 stages
        ws[:4].zero_()
        assert not ws[:256].any()
        if n == 3000:  # a warp of each kind gave up, at its first unit
            same = (got[0] == want[0]).flatten(1).all(1)
            assert same.sum() > n * 0.9
        again = call()
        assert all(torch.equal(a, b) for a, b in zip(want, again))
        assert pl.parallax_workspace_status(ws) == (0, 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_of_two_tokens_to_one_slot(dtype):
    """Two sequences append to the same slots: each 16 bytes there are one token's or
    the other's, every other slot and all of q and r are right."""
    Hq, Hkv, D, ps = 16, 8, 128, 64
    seqs = [(40, 50), (40, 50), (3, 9)]
    kp, vp, table, cu, lens = make_cache(seqs, ps, Hkv, D, dtype, seed=150)
    table[1] = table[0]
    (q, r, k, v), w, _, cs = inputs(83, Hq, Hkv, D, D, dtype, seed=151)
    idx = torch.cat([torch.arange(10, 50), torch.arange(10, 50), torch.arange(6, 9)]).int().cuda()
    fq, fr, fk = pl.parallax_qk_norm_rope(q, r, k, cs, idx, *w)
    before_k, before_v = kp.clone(), vp.clone()
    ws = pl.status_workspace("cuda")
    for _ in range(5):
        qo, ro = pl.parallax_norm_rope_append(q, r, k, v, cs, kp, vp, table, lens, cu, None, *w,
                                              workspace=ws)
        assert torch.equal(qo, fq) and torch.equal(ro, fr)
        for pool, before, x in ((kp, before_k, fk), (vp, before_v, v)):
            part = lambda t: t.contiguous().view(torch.int32).unflatten(-1, (-1, 4))
            got, a, b = part(pool[table[0, 0], 10:50]), part(x[:40]), part(x[40:80])
            assert ((got == a).all(-1) | (got == b).all(-1)).all()
            want = before.clone()
            want[table[0, 0], 10:50] = pool[table[0, 0], 10:50]
            want[table[2, 0], 6:9] = x[80:]
            assert torch.equal(pool, want)
    assert int(ws[:4].view(torch.int32)) == 0
