"""Token log probabilities, entropies and top alternatives (dspark_token_logprobs)
and the emitted tokens of a round (dspark_emitted_tokens) against a plain binary64
computation on the CPU.

Tolerances, u = 2^-24, from the kernel's arithmetic: an exponential 2^y, y = z L - K,
has relative error at most u (|z - m| + 0.7) (the fma's rounding, times ln 2, |y| <=
|z - m| L + 1) + u |z - m| (L = log2 e rounded) + 2u (hardware exp2); sums of sixteen in
chains of at most six additions add 6u; everything after is binary64.  With weights p the
error of lse is at most the weighted mean of these, d = u (2 E|z - m| + 9).  The entropy
ln S - T / S is off by at most d + E[(u (2|z - m| + 9) + 7u)(|z - m| + 1)] (T's products
and sums: one rounding and six more).  Each result is rounded once to binary32."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def dev():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from draft_sampling_verification_w1_amd import dspark
    dspark.lib()
    return dspark


def reference(z, ids, n_top):
    """z [N, V] float64 (numpy), ids [N]; the definition, and the bounds above."""
    N, V = z.shape
    r = {"logprob": np.full(N, np.nan), "entropy": np.full(N, np.nan),
         "top_ids": np.full((N, n_top), -1, np.int64), "top_logprobs": np.full((N, n_top), np.nan),
         "tol": np.zeros(N), "tol_h": np.zeros(N)}
    for i in range(N):
        if not 0 <= ids[i] < V or not np.isfinite(z[i]).any():
            continue
        m = z[i].max()
        live = z[i] > -np.inf
        e = np.exp(z[i] - m)
        s = math.fsum(e)
        lse = m + math.log(s)
        p, gap = e[live] / s, (m - z[i][live])
        r["logprob"][i] = z[i, ids[i]] - lse
        r["entropy"][i] = math.log(s) + math.fsum(p * gap)
        order = np.argsort(-z[i], kind="stable")[:n_top]
        order = order[z[i][order] > -np.inf]
        r["top_ids"][i, :order.size] = order
        r["top_logprobs"][i] = -np.inf
        r["top_logprobs"][i, :order.size] = z[i][order] - lse
        r["tol"][i] = U * (2 * np.sum(p * gap) + 9)
        r["tol_h"][i] = r["tol"][i] + np.sum(p * U * (2 * gap + 16) * (gap + 1))
    return r


def check(got, want):
    g = {k: v.cpu().numpy().reshape(want[k].shape) for k, v in got.items()}
    np.testing.assert_array_equal(g["top_ids"], want["top_ids"])
    for name, tol in (("logprob", want["tol"]), ("entropy", want["tol_h"]),
                      ("top_logprobs", want["tol"][:, None])):
        x, y = g[name].astype(np.float64), want[name]
        np.testing.assert_array_equal(np.isnan(x), np.isnan(y), err_msg=name)
        np.testing.assert_array_equal(np.isneginf(x), np.isneginf(y), err_msg=name)
        fine = np.isfinite(y)
        bound = np.broadcast_to(tol, y.shape)[fine] + U * np.abs(y[fine])
        off = np.abs(x[fine] - y[fine])
        assert (off <= bound).all(), (name, float((off / bound).max()))


def make(N, V, dtype, seed, scale=4.0, kind="normal"):
    import torch
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((N, V), generator=g) * scale
    if kind == "ties":           # few distinct values: the lower index decides
        z = torch.randint(-2, 3, (N, V), generator=g).float()
    elif kind == "rising":       # every entry passes the ones before it
        z = torch.arange(V).float().repeat(N, 1) / 64
    elif kind == "falling":
        z = -torch.arange(V).float().repeat(N, 1) / 64
    elif kind == "front":        # nothing but masked entries first
        z[:, :min(V - 1, 6000)] = -math.inf
    elif kind == "sparse":       # fewer finite entries than alternatives
        z[torch.rand((N, V), generator=g) < 1 - 3 / V] = -math.inf
    elif kind == "sure":         # one entry holds nearly all of the mass
        z[:, V // 2] = 60.0
    elif kind == "wide":
        z = z * 1000
    elif kind == "one_lane":     # the best entries all lie in one thread's group
        z[:, V // 3:V // 3 + 8] += 50
    z = z.to(torch.float32 if dtype == "f32" else torch.bfloat16)
    ids = torch.randint(0, V, (N,), generator=g).to(torch.int32)
    return z, ids


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,V,n_top", [
    (1, 1, 1), (1, 7, 3), (3, 8, 64), (5, 97, 0), (2, 1000, 64), (36, 4096, 5), (7, 4097, 20),
    (1, 151936, 1), (2, 100003, 20), (9, 32001, 33), (2100, 513, 4), (260, 9001, 8)])
def test_sizes(dev, dtype, N, V, n_top):
    z, ids = make(N, V, dtype, 1000 * N + V)
    ids[N // 2:N // 2 + 1] = -1 if N > 2 else ids[N // 2]
    got = dev.token_logprobs(z.cuda(), ids.cuda(), n_top)
    check(got, reference(z.double().numpy(), ids.numpy(), n_top))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["ties", "rising", "falling", "front", "sparse", "sure", "wide", "one_lane"])
@pytest.mark.parametrize("N,V", [(2, 20011), (2050, 300)])
def test_values(dev, dtype, kind, N, V):
    z, ids = make(N, V, dtype, 5, kind=kind)
    got = dev.token_logprobs(z.cuda(), ids.cuda(), 20)
    check(got, reference(z.double().numpy(), ids.numpy(), 20))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_rows_and_ids(dev, dtype):
    """Rows without a finite entry, masked given tokens, ids outside the vocabulary."""
    z, ids = make(8, 5000, dtype, 11)
    z[1] = -math.inf
    z[2, ids[2].item()] = -math.inf
    z[3] = -math.inf
    z[3, 4999] = 1.0
    ids[4], ids[5], ids[6] = -1, 5000, 2 ** 31 - 1
    got = dev.token_logprobs(z.cuda(), ids.cuda(), 3)
    check(got, reference(z.double().numpy(), ids.numpy(), 3))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [1, 3, 6])
def test_row_starts_and_strides(dev, dtype, offset):
    """Rows that start at any element and lie further apart than V; what is
    between them is not read as part of a row."""
    import torch
    z, ids = make(6, 3001, dtype, 21)
    ld = 3001 + 2 * offset
    buf = torch.full((6 * ld + offset + 64,), 1e30, dtype=z.dtype, device="cuda")
    view = buf[offset:offset + 6 * ld].view(6, ld)[:, :3001]
    view.copy_(z)
    got = dev.token_logprobs(view, ids.cuda(), 5)
    check(got, reference(z.double().numpy(), ids.numpy(), 5))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["normal", "ties", "falling", "front", "sparse", "sure"])
@pytest.mark.parametrize("offset", [0, 3])
@pytest.mark.parametrize("V", [40009, 40957])
def test_split_rows(dev, dtype, kind, offset, V):
    """Rows that several workgroups share: splits without a finite entry, masked rows,
    skipped ids, rows that start at any element (40,957: some reach into an eleventh
    step of 4,096, the others leave its split empty)."""
    import torch
    N = 5
    z, ids = make(N, V, dtype, 41, kind=kind)
    z[1] = -math.inf
    z[2, :30000] = -math.inf
    ids[2], ids[3] = 17, V
    ld = V + offset
    view = torch.full((N * ld + offset,), 1e30, dtype=z.dtype, device="cuda")[offset:].view(N, ld)[:, :V]
    view.copy_(z)
    got = dev.token_logprobs(view, ids.cuda(), 20)
    check(got, reference(z.double().numpy(), ids.numpy(), 20))


@pytest.mark.parametrize("V", [3001, 30011])
def test_far_rows(dev, V):
    """Rows whose starts lie 2^32 entries apart."""
    import torch
    ld = 2 ** 32 + 5
    if torch.cuda.mem_get_info()[0] < 2 * (2 * ld + V) + (1 << 30):
        pytest.skip("not enough memory")
    z, ids = make(3, V, "bf16", 51)
    view = torch.empty(2 * ld + V, dtype=torch.bfloat16, device="cuda").as_strided((3, V), (ld, 1))
    view.copy_(z)
    got = dev.token_logprobs(view, ids.cuda(), 5)
    check(got, reference(z.double().numpy(), ids.numpy(), 5))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,live", [(1000, 0), (1000, 1), (1024, 40), (63, 62), (64, 64), (65, 1), (1025, 9)])
def test_few_rows_of_many(dev, dtype, N, live):
    """Most rows are skipped: the others, the first and the last row among them, are
    shared by all workgroups."""
    import torch
    V = 57345
    z, ids = make(N, V, dtype, N + live)
    at = torch.randperm(N, generator=torch.Generator().manual_seed(live))
    at = torch.cat([torch.tensor([N - 1, 0]), at[(at > 0) & (at < N - 1)]])
    ids[at[live:]] = torch.tensor([-1, V])[torch.arange(N - live) % 2].to(torch.int32)
    got = dev.token_logprobs(z.cuda(), ids.cuda(), 6)
    check(got, reference(z.double().numpy(), ids.numpy(), 6))


def test_replayed_graph_and_streams(dev):
    """The call inside a graph, replayed with new inputs between eager calls, and
    on a stream of its own: the eager call's bits."""
    import torch
    z, ids = make(40, 30011, "bf16", 31)
    zd, idd = z.cuda(), ids.cuda()
    ws = dev.logprobs_workspace(40, 30011, 7)
    out = dev.token_logprobs(zd, idd, 7, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dev.token_logprobs(zd, idd, 7, ws=ws, out=out)
    side = torch.cuda.Stream()
    for seed in (32, 33, 34):
        z2, ids2 = make(40, 30011, "bf16", seed)
        zd.copy_(z2)
        idd.copy_(ids2)
        g.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()}
        eager = dev.token_logprobs(zd, idd, 7)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other = dev.token_logprobs(zd, idd, 7)
        side.synchronize()
        for k in got:
            assert torch.equal(got[k].view(torch.int32), eager[k].view(torch.int32)), k
            assert torch.equal(other[k].view(torch.int32), eager[k].view(torch.int32)), k
        check(got, reference(z2.double().numpy(), ids2.numpy(), 7))


def test_replayed_graph_with_other_rows(dev):
    """Replays in which other rows, and other numbers of rows, are looked up."""
    import torch
    z, _ = make(70, 40009, "bf16", 61)
    zd, idd = z.cuda(), torch.zeros(70, dtype=torch.int32, device="cuda")
    out = dev.token_logprobs(zd, idd, 4)
    ws = dev.logprobs_workspace(70, 40009, 4)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dev.token_logprobs(zd, idd, 4, ws=ws, out=out)
    gen = torch.Generator().manual_seed(62)
    for live in (0, 3, 70, 1, 41):
        ids = torch.full((70,), -1, dtype=torch.int32)
        at = torch.randperm(70, generator=gen)[:live]
        ids[at] = torch.randint(0, 40009, (live,), generator=gen).to(torch.int32)
        idd.copy_(ids)
        g.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()}
        eager = dev.token_logprobs(zd, idd, 4)
        for k in got:
            assert torch.equal(got[k].view(torch.int32), eager[k].view(torch.int32)), (live, k)
        check(got, reference(z.double().numpy(), ids.numpy(), 4))


@pytest.mark.parametrize("R,gamma", [(1, 1), (4, 8), (300, 16), (5, 64)])
def test_emitted_tokens(dev, R, gamma):
    import torch
    g = torch.Generator().manual_seed(R)
    tok = torch.randint(0, 1000, (R, gamma), generator=g).to(torch.int32)
    n = torch.randint(0, gamma + 1, (R,), generator=g).to(torch.int32)
    last = torch.randint(0, 1000, (R,), generator=g).to(torch.int32)
    got = dev.emitted_tokens(tok.cuda(), n.cuda(), last.cuda()).cpu()
    want = torch.full((R, gamma + 1), -1, dtype=torch.int32)
    for r in range(R):
        want[r, :n[r]] = tok[r, :n[r]]
        want[r, n[r]] = last[r]
    assert torch.equal(got, want)
