"""The serving operators run together: examples/paged_decode.py decodes with a
paged cache, drafts, grammars and penalties."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("paged_decode", os.path.join(ROOT, "examples", "paged_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("requests,steps", [(1, 5), (6, 20)])
def test_decoding_with_the_paged_cache(example, requests, steps):
    r = example.main(["--requests", str(requests), "--steps", str(steps)])
    # the attended values are rounded to bf16 (2^-8 relative) on both paths, pass
    # through two bf16 products (2^-8 each) and the weights are rounded once more
    # on the cached one: 4 * 2^-8 of the largest logit
    assert r["worst"] < 4 * 2.0 ** -8
    assert r["allowed"]
    d = r["decoder"]
    assert requests * steps <= r["tokens"] <= requests * steps * 8
    assert r["tokens"] == r["accepted"] + requests * steps
    # every page has one owner
    held = [d.table[b, :int(d.owned[b])] for b in range(requests)]
    n, (head, free) = d.ring.numel(), d.ring_state.tolist()
    held.append(d.ring[(head + torch.arange(free, device="cuda")) % n])
    assert torch.equal(torch.sort(torch.cat(held)).values, torch.arange(n, dtype=torch.int32, device="cuda"))
    # the same seed gives the same tokens
    again = example.main(["--requests", str(requests), "--steps", str(steps)])["decoder"]
    assert torch.equal(again.hist, d.hist)
