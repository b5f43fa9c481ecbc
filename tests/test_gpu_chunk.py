"""GPU tests of the chunk attention over a paged cache (parallax_prefill_paged)
against the definition in 64 bits.

Tolerance of an output o_d: half a bf16 step, 2^-8 |o_d|, plus a share of
S_d = sum_i w_i (1 + |s_i| + |s_i - sbar|) (|v_id| + |vbar_d|), the size of the terms
it is summed from: with rounded weights e_i (1 + x_i) and e_i s_i (1 + x_i) (1 + y_i),
and l, b summed from them, o = sum_i w_i (v_i - vbar) (1 + s_i - sbar) moves by x_i
times its term (1 + s_i - sbar) and by y_i times w_i s_i (v_i - vbar), the uncentred
score. The share: x and y are fp16 roundings, 2^-12 each, 4.9e-4; the scores' error (8 accumulation steps of 2^-23 over sums that
reach 10 in the exponent and 80 in s), 1.2e-5 + 8e-5; and the value products'
accumulator, off by at most 2^-23 a step of 16 keys, of which every term passes
n / 16, 8e-9 n. 7e-4 + 6e-8 n covers them at n keys (the hi + lo weights of keys
whose values do not fit fp16 are closer, but take four times the steps)."""
import pytest
import torch

import oracle
from parameterized_local_linear_b200 import binding as pl
from test_gpu_norm_rope import inputs as rope_inputs
from test_gpu_norm_rope import make_cache

pytestmark = pytest.mark.gpu


def reference(q, r, kp, vp, table, cu, lens, causal, scale):
    """(o, S) in fp64, row by row from the definition; untouched rows stay NaN."""
    G = q.shape[1] // kp.shape[2]
    ps, D = kp.shape[1], q.shape[2]
    o = torch.full(q.shape, float("nan"), dtype=torch.float64, device="cuda")
    S = torch.zeros_like(o)
    for b in range(len(lens)):
        a, e, n = int(cu[b]), int(cu[b + 1]), int(lens[b])
        if e == a:
            continue
        i = torch.arange(n, device="cuda")
        page = table[b].long()[i // ps]
        ok = (page >= 0) & (page < kp.shape[0])
        page = page.clamp(0, kp.shape[0] - 1)
        k, v = (torch.where(ok[:, None, None], x[page, i % ps].double(), 0.0)
                .repeat_interleave(G, 1).transpose(0, 1) for x in (kp, vp))  # [Hq, n, D]
        qq = q[a:e].double().transpose(0, 1)
        c = e - a
        seen = ok[None, :] & (i[None, :] <= (torch.arange(c, device="cuda") + n - c)[:, None]
                              if causal else torch.ones(c, n, device="cuda", dtype=torch.bool))
        t = (qq @ k.transpose(1, 2) * scale).masked_fill(~seen, float("-inf"))
        w = torch.softmax(t, -1).nan_to_num(0.0)
        vbar = w @ v
        s = torch.zeros_like(w) if r is None else r[a:e].double().transpose(0, 1) @ k.transpose(1, 2)
        dev = s - (w * s).sum(-1, keepdim=True)
        o[a:e] = (vbar + (w * dev) @ v - (w * dev).sum(-1, keepdim=True) * vbar).transpose(0, 1)
        ww = w * (1 + s.abs() + dev.abs())
        S[a:e] = (ww @ v.abs() + ww.sum(-1, keepdim=True) * vbar.abs()).transpose(0, 1)
    return o, S


def check(got, o, S, nmax, what=()):
    assert got.dtype == torch.bfloat16
    rows = ~o.isnan().all(-1).all(-1)
    err = (got.double() - o).abs()[rows]
    tol = (2.0 ** -8 * o.abs() + (7e-4 + 6e-8 * nmax) * S)[rows]
    bad = ~(err <= tol)
    assert not bad.any(), (what, err[bad].max().item(), (err / tol.clamp_min(1e-30)).max().item())


def make(seqs, ps, Hq, Hkv, D, seed, pad=0, poison=True, r_scale=0.5):
    kp, vp, table, cu, lens = make_cache(seqs, ps, Hkv, D, torch.bfloat16, seed)
    n = int(cu[-1]) + pad
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn(max(n, 1), Hq, D, device="cuda", generator=g).bfloat16()
    r = (torch.randn(max(n, 1), Hq, D, device="cuda", generator=g) * r_scale).bfloat16()
    if poison:  # every slot that no key fills
        used = torch.zeros(kp.shape[:2], dtype=torch.bool)
        for b, (_, m) in enumerate(seqs):
            i = torch.arange(m)
            used[table[b].cpu().long()[i // ps], i % ps] = True
        kp[~used.cuda()] = float("nan")
        vp[~used.cuda()] = float("nan")
    return q, r, kp, vp, table, cu, lens


SHAPES = [
    [(1, 1)],
    [(1, 64)],
    [(2, 65), (64, 64), (1, 63)],
    [(5, 5), (0, 70), (130, 200), (0, 0), (1, 129), (65, 300)],
    [(3, 700), (200, 1000)],
    [(1, 130)] * 40,
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,Hq,Hkv", [(128, 16, 8), (128, 2, 2), (64, 8, 2), (64, 3, 1)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_matches_definition(shape, D, Hq, Hkv, causal):
    seqs = SHAPES[shape]
    q, r, kp, vp, table, cu, lens = make(seqs, 64 if shape % 2 else 128, Hq, Hkv, D, 70 + shape)
    scale = D ** -0.5
    for probe in (True, False):
        ws = pl.prefill_paged_workspace(len(seqs), q.shape[0], Hq, Hkv, D, q.device)
        got = pl.parallax_prefill_paged(q, r if probe else None, kp, vp, table, lens, cu,
                                        causal=causal, probe=probe, workspace=ws)
        o, S = reference(q, r if probe else None, kp, vp, table, cu, lens, causal, scale)
        check(got, o, S, max(n for _, n in seqs), (seqs, D, probe))
        assert int(ws[:4].view(torch.int32)) == 0
        again = pl.parallax_prefill_paged(q, r if probe else None, kp, vp, table, lens, cu,
                                          causal=causal, probe=probe, workspace=ws)
        assert torch.equal(got, again)


@pytest.mark.parametrize("r_scale", [0.0, 1.0, 2.0])
def test_probe_scales_and_oracle(r_scale):
    seqs = [(33, 150), (4, 4)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 4, 2, 128, 80, r_scale=r_scale)
    got = pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu, scale=0.07)
    o, S = reference(q, r, kp, vp, table, cu, lens, True, 0.07)
    check(got, o, S, 150)
    want = oracle.parallax_prefill_paged(q, r, kp, vp, table, cu, lens, 0.07)
    assert abs(o.cpu().numpy() - want).max() <= 1e-9


@pytest.mark.parametrize("G,D", [(5, 64), (8, 128), (16, 64), (128, 64)])
def test_large_and_odd_groups(G, D):
    seqs = [(3, 70), (140, 260), (1, 1)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 2 * G, 2, D, 85)
    got = pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu)
    o, S = reference(q, r, kp, vp, table, cu, lens, True, D ** -0.5)
    check(got, o, S, 260, G)


def test_long_context_is_split_and_merged():
    """One kv head, few rows: every CTA holds a part of each item."""
    for seqs in ([(4, 20000)], [(64, 9001)], [(300, 5000), (1, 12345)]):
        q, r, kp, vp, table, cu, lens = make(seqs, 256, 2, 1, 128, 90)
        got = pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu)
        o, S = reference(q, r, kp, vp, table, cu, lens, True, 128 ** -0.5)
        check(got, o, S, max(n for _, n in seqs), seqs)


def test_large_scores_and_offsets():
    """Keys with a common offset (large s and t with small spread) and logits
    that grow along the row, so that the running maximum is rescaled often."""
    seqs = [(40, 400)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 4, 2, 64, 95, poison=False)
    i = torch.arange(400, device="cuda")
    page, slot = table[0].long()[i // 64], i % 64
    kp[page, slot] = (kp[page, slot].float() * (0.02 * i[:, None, None] + 0.1) + 1.0).bfloat16()
    got = pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu, scale=0.5)
    o, S = reference(q, r, kp, vp, table, cu, lens, True, 0.5)
    # scores up to 40 times those of the tolerance's derivation, and so their error
    err = (got.double() - o).abs()
    assert (err <= 2.0 ** -8 * o.abs() + 40 * 7e-4 * S).all()


@pytest.mark.parametrize("D", [64, 128])
def test_value_and_probe_ranges(D):
    """Blocks of 16 keys whose values leave fp16's range or are tiny, next to
    blocks that fit; probe rows from 2^-40 to scores of 2^17, changing along the keys."""
    seqs = [(50, 230), (130, 330)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 4, 2, D, 96)
    i = torch.arange(330, device="cuda")
    page, slot = table[1].long()[i // 64], i % 64
    base_v, base_k = vp.clone(), kp.clone()
    ws = pl.prefill_paged_workspace(2, q.shape[0], 4, 2, D, q.device)

    def run(what, rr=r):
        ws.zero_()
        got = pl.parallax_prefill_paged(q, rr, kp, vp, table, lens, cu, workspace=ws)
        o, S = reference(q, rr, kp, vp, table, cu, lens, True, D ** -0.5)
        check(got, o, S, 330, what)
        assert int(ws[:4].view(torch.int32)) == 0

    for what, scale in (("large", 1e6), ("above fp16", 7e4 / 3), ("tiny", 1e-5), ("zero", 0.0)):
        vp.copy_(base_v)
        vp[page[48:80], slot[48:80]] = (base_v[page[48:80], slot[48:80]].float() * scale).bfloat16()
        run(what)
    vp.copy_(base_v)
    vp[page[200], slot[200], 1, 3] = 65280.0  # the largest bf16 below 2^16
    run("edge")
    vp[page[200], slot[200], 1, 3] = 65536.0
    run("single")
    vp.copy_(base_v)
    for e in (-40, 3, 10):  # |s| about 8 x 2^e
        run(e, (r.float() * 2.0 ** e).bfloat16())
    # |s| grows and shrinks by 2^12 along the keys, and t with it
    f = torch.ones(330, device="cuda")
    f[100:140], f[300:310] = 64.0, 2.0 ** -6
    kp[page, slot] = (base_k[page, slot].float() * f[:, None, None]).bfloat16()
    got = pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu, scale=D ** -0.5 / 64)
    o, S = reference(q, r, kp, vp, table, cu, lens, True, D ** -0.5 / 64)
    check(got, o, S, 330, "growing")


def test_rows_without_keys_padding_and_bad_pages():
    seqs = [(6, 4), (3, 0), (2, 130), (70, 100)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 4, 2, 128, 97, pad=11)
    out = torch.full_like(q, 5.0)
    ws = pl.prefill_paged_workspace(4, q.shape[0], 4, 2, 128, q.device)
    run = lambda t, n, c=cu: pl.parallax_prefill_paged(q, r, kp, vp, t, n, c, out=out, workspace=ws)
    run(table, lens)
    o, S = reference(q, r, kp, vp, table, cu, lens, True, 128 ** -0.5)
    check(out, o, S, 130)
    assert (out[:2] == 0).all() and (out[6:9] == 0).all()  # no key seen
    assert (out[int(cu[-1]):] == 5).all()                  # rows past the last sequence
    assert int(ws[:4].view(torch.int32)) == 2              # more new tokens than keys
    # a page outside the pool is left out
    for bad in (-1, kp.shape[0], 2 ** 31 - 1):
        t = table.clone()
        t[3, 0] = bad
        ws.zero_()
        run(t, lens)
        o, S = reference(q, r, kp, vp, t, cu, lens, True, 128 ** -0.5)
        check(out, o, S, 130, bad)
        assert int(ws[:4].view(torch.int32)) == 2
    # a length past the table, a negative one: clamped
    n2 = lens.clone()
    n2[2], n2[0] = 10 ** 6, -5
    kp2, vp2 = kp.nan_to_num(0.5), vp.nan_to_num(0.5)
    t = table.clamp_min(0)
    ws.zero_()
    pl.parallax_prefill_paged(q, r, kp2, vp2, t, n2, cu, out=out, workspace=ws)
    fixed = n2.clamp(0, 64 * t.shape[1])
    o, S = reference(q, r, kp2, vp2, t, cu, fixed, True, 128 ** -0.5)
    check(out, o, S, 256)
    assert int(ws[:4].view(torch.int32)) == 2


def test_malformed_cu_seqlens_stays_in_bounds():
    seqs = [(10, 70), (20, 90), (5, 40)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 4, 2, 64, 98, poison=False)
    ws = pl.prefill_paged_workspace(3, q.shape[0], 4, 2, 64, q.device)
    bad = torch.tensor([-3, 12, 9, 1000], dtype=torch.int32, device="cuda")
    got = pl.parallax_prefill_paged(q, r, kp, vp, table, lens, bad, workspace=ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) == 2 and got.isfinite().all()


def test_many_ragged_sequences():
    """More sequences than a warp's lanes, some without new tokens, chunks that
    end anywhere in their row tiles."""
    g = torch.Generator().manual_seed(0)
    q = (torch.randint(0, 40, (150,), generator=g) * (torch.rand(150, generator=g) < 0.7)).tolist()
    seqs = [(c, c + int(x)) for c, x in zip(q, torch.randint(0, 300, (150,), generator=g))]
    for causal in (True, False):
        q, r, kp, vp, table, cu, lens = make(seqs, 64, 6, 2, 64, 112)
        got = pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu, causal=causal)
        o, S = reference(q, r, kp, vp, table, cu, lens, causal, 64 ** -0.5)
        check(got, o, S, 340, causal)


def test_shared_pages_and_two_calls_at_once():
    """Two sequences that share their first pages, in two calls on two streams
    with a workspace each."""
    seqs = [(40, 200), (7, 150)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 8, 4, 128, 113, poison=False)
    table[1, :2] = table[0, :2]
    o, S = reference(q, r, kp, vp, table, cu, lens, True, 128 ** -0.5)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [pl.prefill_paged_workspace(2, 47, 8, 4, 128, q.device) for _ in streams]
    outs = [torch.zeros_like(q) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, w, out in zip(streams, ws, outs):
            pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu, out=out, workspace=w, stream=s)
    torch.cuda.synchronize()
    check(outs[0], o, S, 200)
    assert torch.equal(*outs)


def test_pools_past_32_bit_offsets():
    """Keys in pages whose offsets pass 2^31 elements (2^32 bytes) of the pools, and
    the same pages first in a small pool: the append and the attention give the same."""
    Hq, Hkv, D, ps, pages = 4, 2, 128, 64, 140000
    assert (pages - 8) * ps * Hkv * D > 2 ** 31
    (q, r, k, v), w, _, cs = rope_inputs(300, Hq, Hkv, D, D, torch.bfloat16, 114)
    cu = torch.tensor([0, 170, 300], dtype=torch.int32, device="cuda")
    lens = torch.tensor([170, 130], dtype=torch.int32, device="cuda")
    small = torch.tensor([[5, 1, 7], [0, 3, 2]], dtype=torch.int32, device="cuda")
    got = []
    for n, table in ((8, small), (pages, small + pages - 8)):
        kp, vp = (torch.empty(n, ps, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kp[-8:], vp[-8:] = 0, 0
        a, b = pl.parallax_norm_rope_append(q, r, k, v, cs, kp, vp, table, lens, cu, None, *w)
        out = pl.parallax_prefill_paged(a, b, kp, vp, table, lens, cu)
        got.append((a, b, kp[-8:].clone(), vp[-8:].clone(), out))
        del kp, vp
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert got[0][4].abs().sum() > 0


def test_one_token_form_is_the_decode():
    seqs = [(1, 300), (1, 1), (1, 64), (1, 129)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 16, 8, 128, 99, poison=False)
    t = table.clamp_min(0)
    a = pl.parallax_prefill_paged(q, r, kp, vp, t, lens)
    b = pl.parallax_decode_paged(q, r, kp, vp, t, lens)
    assert torch.equal(a, b)
    o, S = reference(q, r, kp, vp, t, cu, lens, True, 128 ** -0.5)
    check(a, o, S, 300)
    check(pl.parallax_prefill_paged(q, r, kp, vp, t, lens, cu), o, S, 300)


def test_streams_and_two_graphs():
    seqs = [(30, 500), (1, 90)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 4, 2, 128, 101)
    want = pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu, stream=s)
    s.synchronize()
    assert torch.equal(want, got)
    graphs = []
    for _ in range(2):
        ws = pl.prefill_paged_workspace(2, q.shape[0], 4, 2, 128, q.device)
        out = torch.zeros_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu, out=out, workspace=ws)
        graphs.append((graph, out, ws))  # a graph's workspace lives as long as the graph
    for graph, *_ in graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(want, out) for _, out, _ in graphs)


def test_a_batch_without_new_tokens_is_left_alone():
    q, r, kp, vp, table, _, lens = make([(3, 70), (2, 9)], 64, 4, 2, 128, 115, poison=False)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 5.0)
    ws = pl.prefill_paged_workspace(2, 5, 4, 2, 128, q.device)
    pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu, out=out, workspace=ws)
    assert (out == 5).all() and int(ws[:4].view(torch.int32)) == 0


def test_a_captured_step_follows_its_lengths():
    """Norm, append and attention of a padded batch in one graph, replayed for
    chunks and lengths that change in place."""
    Hq, Hkv, D, ps, B, n = 8, 4, 128, 64, 3, 90
    kp, vp = torch.zeros(2, 16, ps, Hkv, D, device="cuda").bfloat16().unbind(0)
    (q, r, k, v), w, _, cs = rope_inputs(n, Hq, Hkv, D, D, torch.bfloat16, 116)
    table = torch.arange(15, dtype=torch.int32, device="cuda").view(3, 5).clone()
    cu = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    ws = pl.prefill_paged_workspace(B, n, Hq, Hkv, D, q.device)
    a, b, out = (torch.zeros(n, Hq, D, device="cuda", dtype=torch.bfloat16) for _ in range(3))

    def step(kp, vp, a, b, out, ws):
        pl.parallax_norm_rope_append(q, r, k, v, cs, kp, vp, table, lens, cu, None, *w, q_out=a,
                                     r_out=b, workspace=ws)
        pl.parallax_prefill_paged(a, b, kp, vp, table, lens, cu, out=out, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(kp, vp, a, b, out, ws)
    kp2, vp2, a2, b2, out2, ws2 = (x.clone() for x in (kp, vp, a, b, out, ws))
    done = torch.zeros(B, dtype=torch.int32)
    for chunks in ([40, 30, 20], [1, 0, 70], [1, 1, 1], [0, 85, 5]):
        c = torch.tensor(chunks, dtype=torch.int32)
        done += c
        cu[1:].copy_(c.cumsum(0).int())
        lens.copy_(done)
        q.copy_(q.roll(7, 0)), r.copy_(r.roll(7, 0)), k.copy_(k.roll(7, 0)), v.copy_(v.roll(7, 0))
        graph.replay()
        step(kp2, vp2, a2, b2, out2, ws2)
        m = int(c.sum())
        for x, y in ((kp, kp2), (vp, vp2), (a, a2), (b, b2), (out, out2)):
            assert torch.equal(x, y)
        o, S = reference(a, b, kp, vp, table, cu, lens, True, D ** -0.5)
        check(out[:m], o[:m], S[:m], 200, chunks)
    assert int(ws[:4].view(torch.int32)) == 0


def test_bounded_wait_reports_and_context_survives():
    """The producer never loads the first K tile: the waits run out, the status
    word says so, and the next call is right."""
    import ctypes
    seqs = [(30, 500)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 4, 2, 128, 103)
    ws = pl.prefill_paged_workspace(1, 30, 4, 2, 128, q.device)
    out = torch.zeros_like(q)
    fn = pl.load_library().parallax_testing_prefill_paged_stalled
    i, vp_, f = ctypes.c_int, ctypes.c_void_p, ctypes.c_float
    fn.argtypes = [vp_] * 8 + [i] * 5 + [f, i, vp_] + [i] * 4 + [vp_, ctypes.c_size_t, i]
    fn.restype = i
    rc = fn(q.data_ptr(), r.data_ptr(), kp.data_ptr(), vp.data_ptr(), table.data_ptr(),
            cu.data_ptr(), lens.data_ptr(), out.data_ptr(), 1, 30, 4, 2, 128, 0.1, 1,
            torch.cuda.current_stream().cuda_stream, kp.shape[0], 64, table.shape[1], 1,
            ws.data_ptr(), ws.numel(), 50)
    assert rc == 0
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) & 1
    ws[:256].zero_()
    got = pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu, workspace=ws)
    o, S = reference(q, r, kp, vp, table, cu, lens, True, 128 ** -0.5)
    check(got, o, S, 500)
    assert int(ws[:4].view(torch.int32)) == 0


def test_serving_run_together():
    """Prompts in chunks, then decode steps, through append, chunk attention and
    decode over one pool, against one pass over the whole sequences in 64 bits
    (on the bf16 rows that the norm and rotation gave, which have their own tests)."""
    Hq, Hkv, D, ps, total = 8, 4, 128, 64, [150, 64, 9]
    B = len(total)
    (q, r, k, v), w, _, cs = rope_inputs(sum(total), Hq, Hkv, D, D, torch.bfloat16, 110)
    start = torch.tensor([0, *total]).cumsum(0)[:-1]
    kp, vp, table, _, _ = make_cache([(0, n) for n in total], ps, Hkv, D, torch.bfloat16, 111)
    kp.fill_(float("nan")), vp.fill_(float("nan"))
    pos = torch.cat([torch.arange(n) for n in total]).int().cuda()
    fq, fr, fk = pl.parallax_qk_norm_rope(q, r, k, cs, pos, *w)
    done = [0] * B
    ws = pl.prefill_paged_workspace(B, sum(total), Hq, Hkv, D, q.device)
    out = torch.zeros_like(q[:, :Hq]).contiguous()
    for step in ([70, 1, 8], [79, 62, 0], [1, 1, 1]):
        rows = torch.cat([start[b] + torch.arange(done[b], done[b] + c) for b, c in enumerate(step)]).cuda()
        done = [d + c for d, c in zip(done, step)]
        cu = torch.tensor([0, *step]).cumsum(0).int().cuda()
        lens = torch.tensor(done, dtype=torch.int32, device="cuda")
        one = all(c == 1 for c in step)
        a, b = pl.parallax_norm_rope_append(q[rows], r[rows], k[rows], v[rows], cs, kp, vp, table,
                                            lens, None if one else cu, None, *w)
        out[rows] = pl.parallax_prefill_paged(a, b, kp, vp, table, lens, None if one else cu,
                                              workspace=ws)
    cu = torch.tensor([0, *total]).cumsum(0).int().cuda()
    o = torch.zeros(sum(total), Hq, D, dtype=torch.float64, device="cuda")
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    fkp, fvp = torch.zeros_like(kp), torch.zeros_like(vp)
    for b, n in enumerate(total):
        i = torch.arange(n, device="cuda")
        fkp[table[b].long()[i // ps], i % ps] = fk[int(start[b]):int(start[b]) + n]
        fvp[table[b].long()[i // ps], i % ps] = v[int(start[b]):int(start[b]) + n]
    o, S = reference(fq, fr, fkp, fvp, table, cu, lens, True, D ** -0.5)
    # normed, weighted probe rows: |r| about 1 per dimension and s up to 60
    check(out, o, 3 * S, max(total))


@pytest.mark.parametrize("probe", [True, False])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seqs", [[(7, 90)] * 150, [(3, 3000), (130, 200)]])
def test_small_values_beside_ordinary_ones(seqs, D, probe):
    """Dimensions of V that are small in every key, zero, or far, and single small
    values in rows that a few keys dominate, in blocks whose other values are near 1:
    S_d holds only the dimension's own values, so each has to keep its own bits.
    Whole items (many short sequences) and cut ones."""
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 4, 2, D, 117)
    base = vp.clone()
    f = torch.ones(D, device="cuda")
    f[[3, 4, 5, 6, D - 1]] = torch.tensor([2.0 ** -20, 2.0 ** -30, 2.0 ** -60, 0.0, 2.0 ** 20],
                                          device="cuda")
    g = torch.Generator(device="cuda").manual_seed(118)
    few = torch.rand(vp.shape, device="cuda", generator=g) < 2e-3
    ten = torch.rand(vp.shape, device="cuda", generator=g) < 0.1
    for what, v, scale in (("dims", base.float() * f, D ** -0.5),
                           ("few", torch.where(few, base.float() * 2.0 ** -28, base.float()), 1.0),
                           ("zeros", torch.where(ten, 0.0, base.float()), D ** -0.5),
                           ("small", base.float() * 2.0 ** -24, D ** -0.5)):
        vp.copy_(v)
        got = pl.parallax_prefill_paged(q, r if probe else None, kp, vp, table, lens, cu,
                                        scale=scale, probe=probe)
        o, S = reference(q, r if probe else None, kp, vp, table, cu, lens, True, scale)
        check(got, o, S, 3000, what)


def test_a_nan_among_the_values_is_not_hidden():
    """V below the length has to be finite; a NaN there reaches the rows that see it."""
    q, r, kp, vp, table, cu, lens = make([(2, 70)], 64, 2, 1, 64, 119, poison=False)
    vp[table[0, 0].long(), 20, 0, 7] = float("nan")
    out = pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu)
    assert out[:, :, 7].isnan().all() and out[:, :, :7].isfinite().all()


@pytest.mark.parametrize("D", [64, 128])
def test_far_probe_scores(D):
    """Scores of 2^23 and 2^53 in all keys, and a key of weight 0 whose score is 2^20
    times the others': e s of the others is then off by at most 2^-33 of the largest |s|
    a key, so A and C by 2^-33 |s| sum |v| and their share of vbar."""
    seqs = [(50, 230), (9, 330)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 4, 2, D, 122)
    for e in (20, 50):
        rr = (r.float() * 2.0 ** e).bfloat16()
        got = pl.parallax_prefill_paged(q, rr, kp, vp, table, lens, cu)
        o, S = reference(q, rr, kp, vp, table, cu, lens, True, D ** -0.5)
        check(got, o, S, 330, e)
    q[:], r[:] = 0.25 * q, 0.25 * r  # small scores, so that weights stay near each other
    q[..., 0], r[..., 0], q[..., 1], r[..., 1] = 4.0, 0.0, 0.0, 1.0
    kp[..., 1] = torch.where(kp[..., 1].isnan(), kp[..., 1], kp[..., 1] * 0)
    for b, at in ((0, 5), (1, 100)):
        page, slot = int(table[b, at // 64]), at % 64
        kp[page, slot] = 0
        kp[page, slot, :, 0], kp[page, slot, :, 1] = -2.0 ** 9, 2.0 ** 20
    got = pl.parallax_prefill_paged(q, r, kp, vp, table, lens, cu, scale=0.5)
    o, S = reference(q, r, kp, vp, table, cu, lens, True, 0.5)
    for b, (c, n) in enumerate(seqs):
        i = torch.arange(n, device="cuda")
        page = table[b].long()[i // 64]
        k, v = (x[page, i % 64].double().repeat_interleave(2, 1).transpose(0, 1) for x in (kp, vp))
        rows = slice(int(cu[b]), int(cu[b + 1]))
        t = q[rows].double().transpose(0, 1) @ k.transpose(1, 2) * 0.5
        t = t.masked_fill(i > (torch.arange(c, device="cuda") + n - c)[:, None], float("-inf"))
        w = torch.softmax(t, -1)
        seen = (w > 0).double()
        lost = 2.0 ** -33 * 2.0 ** 20 * w.amax(-1, keepdim=True)
        S[rows] += (lost * (seen @ v.abs() + seen.sum(-1, keepdim=True) * (w @ v).abs())
                    ).transpose(0, 1) / 7e-4
    check(got, o, S, 330, "one")


@pytest.mark.parametrize("G", [1, 4, 8, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_single_tokens_beside_their_decode(G, D):
    """One token per sequence through the tcgen05 kernel (cu_seqlens_q given) and
    through the decode of the same rows, groups of up to 16: both against the
    definition, and their correction c = o - vbar as a whole. bf16 rounding leaves an
    element off by up to 2^-8 |o|, at random: the errors' share of c, <err, c> / <c, c>,
    is then off by 2^-8 / sqrt(3) sqrt(sum o^2 c^2) / sum c^2, five times that at most,
    where a loss of one part in 2^11 of C would show (2^-12 for the weights' roundings)."""
    lens = [1, 2, 63, 64, 65, 129, 300, 777] * 4
    seqs = [(1, n) for n in lens]
    Hkv, Hq = 2, 2 * G
    q, r, kp, vp, table, cu, lens = make(seqs, 64, Hq, Hkv, D, 123, poison=False)
    t = table.clamp_min(0)
    o, S = reference(q, r, kp, vp, t, cu, lens, True, D ** -0.5)
    vbar, _ = reference(q, None, kp, vp, t, cu, lens, True, D ** -0.5)
    c = o - vbar
    slack = 2.0 ** -12 + 5 * 2.0 ** -8 / 3 ** 0.5 * ((o * c).square().sum().sqrt() / c.square().sum())
    for cu_ in (cu, None):
        ws = pl.prefill_paged_workspace(len(seqs), q.shape[0], Hq, Hkv, D, q.device)
        got = pl.parallax_prefill_paged(q, r, kp, vp, t, lens, cu_, workspace=ws)
        check(got, o, S, 777, (G, D, cu_ is None))
        share = ((got.double() - o) * c).sum() / c.square().sum()
        assert abs(share) <= slack, (share, slack)
        assert pl.parallax_workspace_status(ws) == (0, 0)


@pytest.mark.parametrize("probe", [True, False])
@pytest.mark.parametrize("D,G", [(64, 8), (128, 16), (64, 5), (128, 128)])
def test_one_token_form_of_large_groups(D, G, probe):
    """Groups that the decode's TMA kernel has no room for run on the chunk kernel, with
    the results (bit for bit) of the same call with cu_seqlens_q; sequences without
    keys are zeros and no error."""
    seqs = [(1, n) for n in (300, 1, 0, 64, 129, 0, 2000)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 2 * G, 2, D, 124)
    ws = pl.prefill_paged_workspace(len(seqs), len(seqs), 2 * G, 2, D, q.device)
    call = lambda c, causal=True: pl.parallax_prefill_paged(
        q, r if probe else None, kp, vp, table, lens, c, causal=causal, probe=probe, workspace=ws)
    if not probe and G <= 8:  # the decode takes these: values past the lengths are not read
        kp.nan_to_num_(0.5), vp.nan_to_num_(0.5)
        table.clamp_min_(0)
    a = call(None)
    assert pl.parallax_workspace_status(ws) == (0, 0)
    o, S = reference(q, r if probe else None, kp, vp, table, cu, lens, True, D ** -0.5)
    check(a, o, S, 2000, (D, G, probe))
    assert not a[2].any() and not a[5].any()
    if probe or G > 8:
        b = call(cu, causal=False)
        assert pl.parallax_workspace_status(ws) == (0, 0)
        assert torch.equal(a, b) and torch.equal(a, call(None, causal=False))


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("probe", [True, False])
def test_padding_and_broken_rows_stay_among_themselves(probe, bad):
    """Rows of q and r past, before and between the sequences' tokens that are not finite
    (padding that nobody wrote) change no other row, nor does one broken row of a
    sequence, whose own outputs are not finite."""
    seqs = [(5, 200), (70, 300), (1, 64)]
    q, r, kp, vp, table, cu, lens = make(seqs, 64, 6, 2, 128, 125, pad=30)
    q, r = q.roll(10, 0), r.roll(10, 0)
    cu = cu + 10
    o, S = reference(q, r if probe else None, kp, vp, table, cu, lens, True, 128 ** -0.5)
    q[:10], r[:10], q[86:], r[86:] = bad, bad, bad, bad
    q[40, 3], r[41, 2] = bad, bad
    got = pl.parallax_prefill_paged(q, r if probe else None, kp, vp, table, lens, cu, probe=probe)
    assert not got[:10].any() and not got[86:].any()
    broken = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    broken[40, 3], broken[41, 2] = True, probe
    assert not got[broken].isfinite().all(-1).any()
    check(torch.where(broken[..., None], o.bfloat16(), got), o, S, 300)


def test_serving_run_within_the_derived_tolerance(monkeypatch):
    """test_serving_run_together at the tolerance derived at the top of this file, a third
    of its own: the scores of normed, weighted rows (s up to 60) are within those of the
    derivation."""
    whole = check
    monkeypatch.setitem(globals(), "check", lambda got, o, S3, n: whole(got, o, S3 / 3, n))
    test_serving_run_together()
