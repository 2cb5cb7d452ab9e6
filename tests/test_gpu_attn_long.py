"""Sums over long contexts: the tensor core's additions truncate, so a sum that it forms by itself shrinks with its length.

Every request reads the same pages here, so that batches of long contexts stay small; the reference is a plain softmax in
64 bits on the GPU.  Bounds, beside those of tests/attn_util.py (queries are small, so that R, the scores' size, is at
most 1 and their error 2^-17 at most): fp32 adds up 512 tokens on the tensor core, 64 additions each off by at most 2^-23 of
the sum, and those sums in fp32, n / 512 additions off by 2^-24 each; bf16 at most 32768 tokens, 2048 additions."""
import math

import pytest
import torch

import hybrid_linear_attention_causal_b200 as gdn

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
F8 = torch.float8_e4m3fn


class Shared:
    """Requests of `rows` rows over the first kv[n] tokens of one set of pages; values are positive, 0.5 to 2.9."""

    def __init__(self, rows, kv, G, dtype, d=64, ps=128, spread=0.1, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        n, pages = len(kv), -(-max(kv) // ps)
        k = (torch.randn((pages, 1, ps, d), generator=g, device="cuda") * 60).clamp_(-448, 448).to(F8)
        v = (torch.rand((pages, 1, ps, d), generator=g, device="cuda") * 150 + 35).to(F8)
        e = torch.full((pages, 1), -6, dtype=torch.int8, device="cuda")
        self.cache = gdn.AttnCache(k=k.view(torch.uint8), v=v.view(torch.uint8), k_exp=e, v_exp=e.clone())
        self.K, self.V = (x.double().view(-1, d) * 2.0 ** -6 for x in (k, v))
        self.cfg = gdn.AttnConfig(G, 1, d, page_size=ps, dtype=dtype)
        self.q = (torch.randn((n * rows, G, d), generator=g, device="cuda") * spread).to(dtype)
        self.table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(n, 1)
        self.rows, self.kv, self.n, self.d = rows, kv, n, d

    def run(self, verify=False):
        out = torch.empty_like(self.q)
        lens = torch.tensor(self.kv, dtype=torch.int32, device="cuda")
        ws = gdn.alloc_workspace(gdn.attn_extend_workspace_size(self.cfg, self.n, self.q.shape[0]), "cuda")
        if verify:
            gdn.attn_verify(self.cfg, self.q, self.rows, lens, self.table, self.cache, out, ws)
        else:
            cu = torch.arange(self.n + 1, dtype=torch.int32, device="cuda") * self.rows
            gdn.attn_extend(self.cfg, self.q, cu, lens, self.table, self.cache, out, ws)
        torch.cuda.synchronize()
        assert gdn.gdn_get_device_error(ws) == 0
        return out

    def want(self, i, r):
        """Row r of request i, in 64 bits: [G, d]."""
        m = self.kv[i] - self.rows + r + 1
        return torch.softmax(self.q[i * self.rows + r].double() @ self.K[:m].T / math.sqrt(self.d), -1) @ self.V[:m]


SCORES = 2 * math.log(2) * 2.0 ** -17  # what errors of the scores do to a weight and to the sum of the weights


def check_all(s, out):
    """Each element within its bound (values are positive: sums of |p v| are the outputs themselves)."""
    f32 = out.dtype == F32
    for i, kv in enumerate(s.kv):
        for r in range(s.rows):
            ref = s.want(i, r)
            sums = 64 * 2.0 ** -23 + kv / 512 * 2.0 ** -24 if f32 else 2048 * 2.0 ** -23
            rel = (2.0 ** -24 + 2.0 ** -22 if f32 else 2.0 ** -8 + 2.0 ** -11) + SCORES + sums
            worst = ((out[i * s.rows + r].double() - ref).abs() / ref).max().item()
            assert worst <= rel, (i, r, kv, worst / rel)


@pytest.mark.parametrize("rows,G", [(1, 1), (4, 3), (4, 8)])  # one, two and four blocks of 8 rows
@pytest.mark.parametrize("d", [64, 128])
def test_fp32_sums_keep_their_size(rows, G, d):
    s = Shared(rows, [131072 - 37 * i for i in range(512 // rows)], G, F32, d=d, ps=64, seed=rows)
    out = s.run(verify=True)
    s.kv, keep = s.kv[::97], s.q
    out = torch.cat([out[i * rows:(i + 1) * rows] for i in range(0, s.n, 97)])
    s.q = torch.cat([keep[i * rows:(i + 1) * rows] for i in range(0, s.n, 97)])
    check_all(s, out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,G", [(1, 2), (3, 5), (2, 16)])
def test_short_items_around_the_length_that_is_added_up_at_once(dtype, rows, G):
    """Thousands of requests of a step more or less than one, two or three times that many tokens."""
    unit = 512 if dtype == F32 else 4096
    n = 3000 if dtype == F32 else 700
    kv = [unit * (1 + i % 3) + (0, 1, 32, 33, -1, -32, 20)[i % 7] for i in range(n)]
    s = Shared(rows, kv, G, dtype, ps=32, seed=3)
    out = s.run(verify=True)
    some = range(0, n, 29)
    s.q = torch.cat([s.q[i * rows:(i + 1) * rows] for i in some])
    out = torch.cat([out[i * rows:(i + 1) * rows] for i in some])
    s.kv = [kv[i] for i in some]
    check_all(s, out)


def shrink(s, out, picks):
    """The mean relative error of some rows, in the standard deviations of its rounding too."""
    rel = torch.cat([((out[i * s.rows + r].double() - x) / x).flatten() for i, r in picks for x in [s.want(i, r)]])
    return rel.mean().item(), 2.0 ** -8 / math.sqrt(3 * rel.numel())


@pytest.mark.parametrize("n,rows,G,kv", [(1, 40960, 1, 524288 + 40960),  # items of 256 rows
                                         (300, 1, 40, 524288)])         # of 40, whose tiles two streams share
def test_bf16_sums_keep_their_size(n, rows, G, kv):
    """The roundings of many outputs cancel; what is left is the shrinking (0.13 % where 524288 tokens are one sum)."""
    s = Shared(rows, [kv] * n, G, BF, spread=2.5, seed=5)
    out = s.run()
    picks = [(7 * i % n, 641 * i % rows) for i in range(64)]
    mean, sigma = shrink(s, out, picks)
    assert abs(mean) <= 2048 * 2.0 ** -23 + 5 * sigma, mean


@pytest.mark.parametrize("G,rows,unit", [(1, 256, 32768), (40, 1, 65536), (3, 100, 32768)])
def test_items_around_the_tiles_that_are_added_up_at_once(G, rows, unit):
    """One item or two of 256 rows, or one of 40, per request, of 255 to 513 tiles a stream."""
    kv = [unit * (1 + i % 2) + (0, 1, 127, 128, 129, -1, -128, 300)[i % 8] for i in range(170)]
    s = Shared(rows, kv, G, BF, seed=6)
    out = s.run()
    picks = [(i, r) for i in range(0, 170, 3) for r in (0, rows // 2, rows - 1)]
    for i, r in picks:
        ref = s.want(i, r)
        worst = ((out[i * rows + r].double() - ref).abs() / ref).max().item()
        assert worst <= 2.0 ** -8 + 2.0 ** -11 + SCORES + 2048 * 2.0 ** -23, (i, r, kv[i], worst)
