"""Steps in which the pages run out, and what the caller does then."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import gpu_util as gu
from tests import plain_kv
from tests.test_gpu_kv import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    yield


def step_of(context, fresh, rows, page, pages, table, free, count):
    """One step on the GPU, held against the plain plan."""
    step = Step(context, fresh, rows, page, pages, table, free, count)
    step.run()
    want = plain_kv.plan(context, fresh, rows, page, pages, table, free, count)
    step.check(want)
    return want


@pytest.mark.parametrize("end", [False, True])
def test_pages_that_ran_out_are_taken_later(end):
    """Lengths are put back to the first row without a slot (or the request ends); once pages are free again, the tokens come again, and
    every page is held by one request or free, throughout."""
    page, pages, width, rows = 16, 12, 8, 120
    table, free = np.full((4, width), -1, np.int32), np.arange(pages)[::-1].copy()
    # 5 + 3 of 12 pages; then 0 and 2 want 2 and 4 more, of which 4 are there: the second lacks its last two
    plan = step_of(np.zeros(4, int), np.array([70, 0, 40, 0]), rows, page, pages, table, free, pages)
    assert plan["missing"] == 0 and plan["left"] == 4
    free = np.full(pages, -1)
    free[:4] = plan["stack"]
    plan = step_of(np.array(plan["lengths"]), np.array([30, 0, 60, 0]), rows, page, pages, plan["table"], free, 4)
    assert plan["left"] == 0 and plan["missing"] == 20
    lengths = np.array(plan["lengths"])
    for s in range(4):
        for i in range(plan["offsets"][s], plan["offsets"][s + 1]):
            if plan["slots"][i] < 0:
                lengths[s] = plan["positions"][i]
                break
    assert lengths.tolist() == [100, 0, 80, 0]

    def held(table, lengths):
        return [int(p) for s in range(4) for p in table[s, :-(-lengths[s] // page)]]

    assert sorted(held(plan["table"], lengths)) == list(range(pages))
    # the first request ends; the third brings its last 20 tokens again, or ends as well
    fresh = np.array([-1, 0, -1 if end else 20, 0])
    plan = step_of(np.array(plan["lengths"]) if end else lengths, fresh, rows, page, pages, plan["table"], np.full(pages, -1), 0)
    assert plan["missing"] == 0 and plan["lengths"] == [0, 0, 0 if end else 100, 0]
    assert sorted(held(plan["table"], plan["lengths"]) + plan["stack"]) == list(range(pages))
    if not end:
        assert plan["positions"][:20] == list(range(80, 100)) and min(plan["slots"][:20]) >= 0
