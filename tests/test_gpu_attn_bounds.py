"""The 8-bit paged attention on the GPU within bounds taken row by row (tests/attn_util.py), at options, exponents
and magnitudes far from the usual ones."""
import numpy as np
import pytest
import torch

import hybrid_linear_attention_causal_b200 as gdn
from oracle import attn as A
from tests.attn_util import bounds, check_rows, extreme_case
from tests.test_gpu_attn import BF, F32, Case, call, fresh, gpu_append, i32, random_tree, same_cache

pytestmark = pytest.mark.gpu

MODES = [("decode", 1), ("verify", 4), ("tree", 4), ("extend", 0)]


def lens_of(mode, D, n):
    return [90, 1, 30, 7][:n] if mode == "extend" else [D] * n


def attend(c, mode, D, ref=None, **kw):
    """One call and its check; kw: options of `call`, ref: those options under the definition's names."""
    parents = random_tree(c.rng, len(c.kv), D) if mode == "tree" else None
    got = call(c, "verify" if mode == "tree" else mode, D=D, parents=parents, **kw)
    check_rows(c, got, parents=parents, **(ref or {}))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode,D", MODES)
@pytest.mark.parametrize("hq,hkv", [(4, 2), (60, 1)])  # the kernel of split tokens (extend aside) and that of tiles
@pytest.mark.parametrize("cap", [1e-39, 0.5, 256.0, 257.0, 1e4, 1e6, 1e30, 3e38])
def test_caps_of_any_size(dtype, mode, D, hq, hkv, cap):
    """A cap far above the scores changes nothing, and one far below them makes them equal in size: the error does not
    grow with the cap."""
    c = Case(lens_of(mode, D, 4), [700, 20, 130, 257], hq, hkv, 128 if hq == 4 else 64, 32, dtype, seed=51)
    c.q[0, 1] = 0.0
    attend(c, mode, D, dict(cap=cap), logit_cap=cap)
    attend(c, mode, D, dict(cap=cap, window=100, slopes=[0.1] * hq), logit_cap=cap, window=100, slopes=[0.1] * hq)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode,D", MODES)
@pytest.mark.parametrize("hq,hkv", [(4, 2), (60, 1)])
@pytest.mark.parametrize("power", [123, 80, -80, -118])
def test_queries_of_any_magnitude(dtype, mode, D, hq, hkv, power):
    """Queries at both ends of their type's range, under a scale that brings the scores back to ordinary ones."""
    c = Case(lens_of(mode, D, 3), [300, 20, 130], hq, hkv, 64 if hq == 4 else 128, 16, dtype, seed=52,
             qscale=1.5 * 2.0 ** power)
    scale = 0.1 * 2.0 ** -power
    attend(c, mode, D, dict(scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode,D", MODES)
@pytest.mark.parametrize("hq", [4, 100])
def test_exponents_far_apart(dtype, mode, D, hq):
    attend(extreme_case(Case, lens_of(mode, D, 2), dtype, hq), mode, D)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,L,hq,hkv", [(256, 2, 16, 2), (700, 2, 6, 2), (300, 8, 2, 2)])
def test_short_extends_are_verified_drafts(dtype, n, L, hq, hkv):
    """Many requests of few rows each: attn_extend and attn_verify take the same kernel, and give the same bits."""
    rng = np.random.default_rng(53)
    c = Case([L] * n, [int(x) for x in rng.integers(L, 150, n)], hq, hkv, 64, 32, dtype, seed=53)
    got = call(c, "extend")
    check_rows(c, got)
    for a, b in zip(got, call(c, "verify", D=L)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("opts", [{}, dict(cap=20.0, window=70, slopes=[0.5 / (h + 1) for h in range(8)])])
def test_long_requests_among_many_short_ones(dtype, d, opts):
    """Requests on both sides of the rows at which the kernels change, with padding, lengths too short and too long,
    requests without rows and rows behind the last request among them, on either side."""
    rng = np.random.default_rng(54)
    G, n = 4, 200
    lens = [1] * n
    for i, rows in ((3, 7), (50, 8), (51, 9), (52, 0), (90, 40), (91, 40), (92, 8), (120, 8), (150, 300), (199, 130)):
        lens[i] = rows
    kv = [int(max(l, x)) for l, x in zip(lens, rng.integers(1, 200, n))]
    kv[150], kv[199], kv[60], kv[52] = 900, 130, 777, 30
    c = Case(lens, kv, 2 * G, 2, d, 16, dtype, seed=54)
    T = sum(lens)
    q = torch.cat([c.q, c.q[:9]]).cuda()
    out = torch.full((T + 9, c.hq, c.d), 7.0, dtype=dtype, device="cuda")
    names = dict(cap="logit_cap")
    kw = {names.get(k, k): v for k, v in opts.items()}
    got, lse = call(c, "extend", q=q, out=out.clone(), **kw)
    check_rows(c, (got[:T], lse[:T]), **opts)
    assert (got[T:] == 7.0).all() and torch.isnan(lse[T:]).all()
    c.kv[90], c.kv[7] = -1, 0                   # padding: 160 rows per key, and 4
    c.kv[91], c.kv[92] = 39, 7                  # shorter than their rows
    c.kv[120] = c.mp * c.ps + 1                 # longer than the table
    again, lagain = call(c, "extend", q=q, out=out, want_err=gdn.GDN_DEVERR_KV_LEN, **kw)
    first = np.concatenate([[0], np.cumsum(lens)])
    for i in (90, 7, 91, 92, 120):
        rows = slice(first[i], first[i + 1])
        assert not again[rows].any() and torch.isneginf(lagain[rows]).all()
    keep = np.repeat([i not in (90, 7, 91, 92, 120) for i in range(n)], lens)
    c.kv = [-1 if i in (91, 92, 120) else x for i, x in enumerate(c.kv)]
    check_rows(c, (again[:T], lagain[:T]), **opts)
    assert keep.sum() == T - 97


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("D,G", [(1, 16), (1, 17), (2, 8), (1, 32), (1, 33), (4, 8), (3, 11)])
def test_rows_per_key_where_the_kernels_change(dtype, d, D, G):
    c = Case([D] * 5, [300, D, 0, 64, 129], G, 1, d, 32, dtype, seed=58)
    attend(c, "verify", D)


def test_a_mixed_batch_captured():
    """A captured extend whose lengths change place: the long request becomes short, and a short one long."""
    lens = [[600, *[1] * 99], [*[1] * 70, 590, *[1] * 20, 10, *[0] * 8]]
    cases = [Case(x, [max(y, 1) + 40 for y in x], 8, 2, 64, 16, BF, seed=55, extra_pages=3) for x in lens]
    T = max(sum(x) for x in lens)
    cfg = cases[0].cfg()
    ws = gdn.alloc_workspace(gdn.attn_extend_workspace_size(cfg, 100, T), "cuda")
    pages = max(c.np["k"].shape[0] for c in cases)
    cache = gdn.alloc_attn_cache(cfg, pages, "cuda")
    mp = max(c.mp for c in cases)
    q, out = (torch.zeros((T, 8, 64), dtype=BF, device="cuda") for _ in range(2))
    cu, kv, table = (torch.zeros(x, dtype=torch.int32, device="cuda") for x in ((101,), (100,), (100, mp)))
    run = lambda: gdn.attn_extend(cfg, q, cu, kv, table, cache, out, ws)

    def load(c):
        t = sum(c.lens)
        q[:t].copy_(c.q)
        cu.copy_(i32(np.concatenate([[0], np.cumsum(c.lens)])))
        kv.copy_(i32(c.kv))
        table[:, :c.mp].copy_(torch.from_numpy(c.table))
        for name in ("k", "v", "k_exp", "v_exp"):
            x = torch.from_numpy(c.np[name])
            getattr(cache, name)[:x.shape[0]].copy_(x)

    load(cases[0])
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for c in (cases[1], cases[0]):
        load(c)
        g.replay()
        torch.cuda.synchronize()
        assert gdn.gdn_get_device_error(ws) == 0
        ref, _, tol, _ = bounds(c)
        got = out[:sum(c.lens)].cpu().double().numpy()
        assert (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_a_rejected_draft_leaves(dtype):
    """Outliers appended as drafts and replaced: the exponent they raised stays, earlier tokens of their page are off by up to
    half its smallest step, pages before and after are as if the drafts had never been, and so is the page once it is
    appended again from its first token."""
    rng = np.random.default_rng(56)
    ps, hkv, d = 16, 2, 64
    cfg = gdn.AttnConfig(hkv, hkv, d, page_size=ps, dtype=dtype)
    ws = gdn.alloc_workspace(gdn.attn_append_workspace_size(cfg, 1, 40), "cuda")
    table = i32([[3, 0, 2, 1]])
    x = torch.from_numpy(rng.standard_normal((40, hkv, d))).to(dtype)

    def put(cache, rows, start):
        gdn.attn_append(cfg, cache, rows.cuda(), rows.cuda(), None, i32([start]), table, ws)

    caches = [gdn.alloc_attn_cache(cfg, 4, "cuda") for _ in range(2)]
    for i, cache in enumerate(caches):
        put(cache, x[:21], 0)
        if i:
            put(cache, x[21:33] * 1e4, 21)  # the drafts: pages 1 and 2 of the request
        put(cache, x[21:40], 21)
    torch.cuda.synchronize()
    clean, after = ({n: getattr(c, n).cpu().numpy() for n in ("k", "v", "k_exp", "v_exp")} for c in caches)
    assert gdn.gdn_get_device_error(ws) == 0
    for n in "kv":
        assert np.array_equal(clean[n][[3, 2]], after[n][[3, 2]])
        assert np.array_equal(clean[n + "_exp"][[3, 2]], after[n + "_exp"][[3, 2]])
        e = after[n + "_exp"][0].astype(float)
        assert (e > clean[n + "_exp"][0]).all()
        old, new = (A.CODE[c[n][0, :, :5]] * 2.0 ** c[n + "_exp"][0].astype(float)[:, None, None] for c in (clean, after))
        assert (np.abs(new - old) <= 2.0 ** (e[:, None, None] - 10)).all() and (new != old).any()
    put(caches[1], x[16:40], 16)
    put(caches[0], x[16:40], 16)
    torch.cuda.synchronize()
    for n in ("k", "v", "k_exp", "v_exp"):
        assert torch.equal(*(getattr(c, n) for c in caches))


@pytest.mark.parametrize("hq", [4, 40])
def test_lengths_of_requests_without_rows(hq):
    """They raise nothing, wherever they point, in any call; the same lengths with a row do."""
    c = Case([2, 0, 3, 0], [20, 30, 40, 50], hq, 2, 64, 16, BF, seed=57)
    good = call(c, "extend")
    c.kv[1], c.kv[3] = 16 * c.mp + 1, 2 ** 31 - 1
    for a, b in zip(call(c, "extend"), good):
        assert torch.equal(a, b)
    c.kv[2] = 16 * c.mp + 1
    call(c, "extend", want_err=gdn.GDN_DEVERR_KV_LEN)
    rng = np.random.default_rng(57)
    ref = fresh(4, 2, 16, 64, rng)
    cache = gdn.AttnCache(**{n: torch.from_numpy(x.copy()).cuda() for n, x in ref.items()})
    x = torch.from_numpy(rng.standard_normal((2, 2, 64))).to(BF)
    gpu_append(x.cuda(), x.cuda(), [0, 0, 2], [2 ** 31 - 1, 5], [[0], [3]], cache, BF, 16, 2, 64)
    A.append(ref, x.double().numpy(), x.double().numpy(), [0, 2], [0, 5], [[0], [3]], 16)
    same_cache(cache, ref)
