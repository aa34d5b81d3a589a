"""Attention over a paged cache: arguments outside the contract that reach nothing beside the outputs, and paths that only
sizes beyond the ordinary take."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import ternary_weight_int8_tb_amd as tb
from tests import gpu_util as gu
from tests.test_gpu_attn_paged import KINDS, Case, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    yield


class Guarded:
    """A tensor within a larger one, with 64 KB of 0x3C on either side."""

    EDGE = 65536

    def __init__(self, like):
        n = like.numel() * like.element_size()
        self.all = torch.full((n + 2 * self.EDGE,), 0x3C, dtype=torch.uint8, device=gu.DEV)
        self.t = self.all[self.EDGE:self.EDGE + n].view(like.dtype).view(like.shape)
        self.t.copy_(like)

    def whole(self):
        return bool((self.all[:self.EDGE] == 0x3C).all() and (self.all[-self.EDGE:] == 0x3C).all())


def guarded_run(c):
    """Runs a case with out and ws guarded; nothing beside them has changed."""
    out, ws = Guarded(c.out), Guarded(c.ws)
    c.out, c.ws = out.t, ws.t
    kept = {n: getattr(c, n).clone().view(torch.uint8) for n in ("dq", "dk", "dv", "dt", "do", "dl")}
    c.run()
    torch.cuda.synchronize()
    assert out.whole() and ws.whole()
    for n, was in kept.items():
        assert torch.equal(getattr(c, n).view(torch.uint8), was), n


@pytest.mark.parametrize("rows,cache", KINDS)
@pytest.mark.parametrize("offsets,lengths", [([0, 100, 2, 2 ** 31 - 1], [40, 50, 60]), ([-5, 3, -2, 9], [40, -50, 2 ** 31 - 1]),
                                             ([12, 0, 12, 0], [1, 2, 3]), ([2 ** 31 - 1, -2 ** 31, 5, 6], [10 ** 9, 50, 60])])
def test_offsets_that_descend(rows, cache, offsets, lengths):
    """Nothing is written."""
    c = Case([(40, 4), (50, 4), (60, 4)], 4, 2, 64, 16, rows, cache, seed=10).upload(extra=2)
    c.do, c.dl = ints(offsets), ints(lengths)
    guarded_run(c)
    assert torch.all(c.out == 77.0)


@pytest.mark.parametrize("rows,cache", KINDS)
def test_offsets_outside_the_rows(rows, cache):
    """Offsets that do not descend count as the nearest row: requests before and behind the rows have none."""
    c = Case([(40, 4), (50, 4), (60, 4)], 4, 2, 64, 16, rows, cache, seed=10).upload(extra=2)
    c.do = ints([-7, 4, 8, 2 ** 31 - 1])       # as [0, 4, 8, 14]
    guarded_run(c)
    first, got = c.out[:8].clone(), c.out[8:].clone()
    c.do = ints([0, 4, 8, 14])
    c.dq = torch.where(torch.isnan(c.dq), torch.zeros_like(c.dq), c.dq)
    c.out.fill_(77.0)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(c.out[:8], first) and torch.equal(c.out[8:12], got[:4])
    # one row for each request, as in decoding, and then rows of none
    d = Case([(40, 1), (50, 1), (60, 1), (9, 1), (0, 0)], 4, 2, 64, 16, rows, cache, seed=11).upload(extra=1)
    d.do = ints([-1, 1, 2, 3, 2 ** 31 - 1, 2 ** 31 - 1])
    guarded_run(d)
    first = d.out[:3].clone()
    d.do = ints([0, 1, 2, 3, 3, 3])
    d.out.fill_(77.0)
    d.run()
    torch.cuda.synchronize()
    assert torch.equal(d.out[:3], first) and torch.all(d.out[3:] == 77.0)


@pytest.mark.parametrize("requests,tokens", [(4096, 65536), (4096, 4096), (64, 64)])
def test_requests_that_all_claim_all_rows(requests, tokens):
    """Together more units than 31 bits count, if each were taken at its word."""
    heads, kv, dim, width, page = 16, 2, 64, 1024, 16
    q = torch.randn(tokens, heads, dim, device=gu.DEV).to(torch.bfloat16)
    k = torch.randn(3, kv, page, dim, device=gu.DEV).to(torch.bfloat16)
    cache = tb.KvCache(k, k.clone())
    table = torch.zeros(requests, width, dtype=torch.int32, device=gu.DEV)
    offsets = ints(np.where(np.arange(requests + 1) % 2 == 1, tokens, 0))
    lengths = ints(np.full(requests, 2 ** 31 - 1))
    out = Guarded(torch.full_like(q, 77.0))
    ws = Guarded(torch.zeros(tb.tb_attn_paged_workspace_bytes(cache, heads, q.dtype, requests, tokens), dtype=torch.uint8, device=gu.DEV))
    tb.tb_attn_paged(q, cache, table, offsets, lengths, 0.125, out.t, ws.t)
    torch.cuda.synchronize()
    assert out.whole() and ws.whole() and torch.all(out.t == 77.0)


@pytest.mark.parametrize("rows,cache", KINDS)
@pytest.mark.parametrize("requests,group,dim,kv", [
    ([(300, 1)] * 3, 40, 64, 1), ([(70, 1), (0, 0), (41, 1)] * 9, 64, 64, 1), ([(65, 1)] * 9, 128, 128, 1), ([(40, 1)] * 17, 33, 256, 2),   # decodes
    ([(33, 1)] * 40 + [(150, 60)], 3, 128, 2), ([(90, 5)], 8, 256, 2), ([(64, 2)] * 12, 4, 64, 1), ([(20, 0)] * 50 + [(50, 50)], 8, 64, 1)])
def test_either_kernel(rows, cache, requests, group, dim, kv):
    """Decodes with more heads than a tile has rows, few and many; chunks beside decodes and beside requests that wait."""
    print(f"either kernel {len(requests)} requests group={group} dim={dim} {rows}/{cache}", flush=True)
    c = Case(requests, group * kv, kv, dim, 16, rows, cache, seed=group)
    c.upload()
    guarded_run(c)
    c.check()


def test_one_workspace_for_a_programs_steps():
    """A workspace of the largest step serves the smaller ones, decodes and chunks."""
    steps = [[(60, 1)] * 40, [(90, 30)], [(33, 3), (70, 1)], [(50, 1)]]
    sized = False
    for requests in steps:
        c = Case(requests, 16, 2, 64, 16, "bf16", "bf16", seed=len(requests)).upload()
        if not sized:
            ws = Guarded(torch.zeros(tb.tb_attn_paged_workspace_bytes(c.handle, 16, torch.bfloat16, 40, 40), dtype=torch.uint8, device=gu.DEV))
            sized = True
        c.ws = ws.t
        c.run().check()
        assert ws.whole()


def test_whole_numbers_past_32_bits():
    """A window, a page size or a number of experts that 32 bits do not hold is refused, not cut off."""
    c = Case([(40, 4)], 4, 2, 64, 16, "bf16", "bf16", seed=14).upload()
    n = 2 ** 32
    refused = [lambda: tb.tb_attn_paged(c.dq, c.handle, c.dt, c.do, c.dl, c.scale, c.out, c.ws, window=n),
               lambda: tb.tb_attn_paged(c.dq, c.handle, c.dt, c.do, c.dl, c.scale, c.out, c.ws, window=n + 5),
               lambda: tb.Rope(torch.zeros(32, dtype=torch.float64, device=gu.DEV), layout=n + 1)]
    one, two = ints([1]), ints([0, 0])
    table, rows = torch.zeros(1, 4, dtype=torch.int32, device=gu.DEV), torch.zeros(1, dtype=torch.int32, device=gu.DEV)
    refused.append(lambda: tb.tb_kv_plan(ints([0]), ints([1]), n + 16, 8, table, ints(np.arange(8)), ints([8]), ints([0]), two, rows, rows.clone(),
                                         ints([0]), ints([0])))
    y = torch.zeros(2, 128, device=gu.DEV)
    refused.append(lambda: tb.tb_moe_combine(y, torch.ones(1, 2, device=gu.DEV), torch.zeros(1, 2, dtype=torch.int32, device=gu.DEV), n + 4,
                                             torch.zeros(1, 128, device=gu.DEV)))
    for call in refused:
        with pytest.raises(tb.TbError) as e:
            call()
        assert e.value.status == tb.TB_EINVAL
    assert tb.tb_attn_paged_workspace_bytes(c.handle, 4, torch.bfloat16, n + 1, n + 4) == 0
    assert torch.all(c.out == 77.0)


@pytest.mark.parametrize("rows,cache", [("f32", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("dim,requests", [(256, [(20000, 1)]), (128, [(40000, 1)]), (64, [(70000, 1)]),
                                          (256, [(30, 1)] * 9 + [(20000, 1)] + [(17, 1)] * 10), (128, [(9, 1)] * 40 + [(9000, 1)])])
def test_units_of_hundreds_of_parts(rows, cache, dim, requests):
    """A unit's parts in more trips of the join than one; the last third of the keys has values of its own, so that no part
    can be left out."""
    print(f"parts dim={dim} {[n for n, _ in requests if n > 99]} {rows}/{cache}", flush=True)
    c = Case(requests, 2, 1, dim, 64, rows, cache, seed=dim)
    s = max(range(len(requests)), key=lambda r: requests[r][0])
    held = -(-c.lengths[s] // 64)
    third = c.table[s, 2 * held // 3:held - 1]
    c.v[third] += 3.0
    c.k[third] *= 0.5
    c.upload()
    guarded_run(c)
    c.check()


@pytest.mark.parametrize("rows,cache", KINDS)
@pytest.mark.parametrize("n,dim", [(300, 64), (700, 64), (300, 128), (600, 256)])
def test_many_ragged_requests_of_several_tokens(n, dim, rows, cache):
    """The kernel for many rows with hundreds of requests, some of them empty: each workgroup finds its own among them."""
    print(f"many ragged {n} dim={dim} {rows}/{cache}", flush=True)
    rng = np.random.default_rng(n + dim)
    new = rng.choice([0, 0, 1, 2, 5, 9], n)
    requests = [(int(m + x) if m else int(x), int(m)) for m, x in zip(new, rng.integers(0, 25, n))]
    requests[n // 3] = (333, 130)
    requests[n - 1] = (0, 0)
    assert sum(m for _, m in requests) > n + 128
    c = Case(requests, 2, 2, dim, 16, rows, cache, seed=n)
    c.upload(extra=1)
    guarded_run(c)
    c.check()
    assert torch.all(c.out[c.tokens:] == 77.0)
