"""GPU: 8-bit AdamW lists of 16.8 million elements and more, whose workgroups take 8192 elements each."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_amd import binding as B
from oracle import adamw as oadam
from tests.gpu_util import say
from tests.test_gpu_adamw import BF16, F32, HY, _check, _lists, _np, _snap

pytestmark = pytest.mark.gpu

SIZES = [1, 8191, 0, 16_900_001, 2049, 8192, 8193, 0, 127, 24577, 6145]
LARGE = 3


def _part(d, j, a, b):
    """Elements a .. b of tensor j, as the list [.., tensor j] that the check of whole tensors takes."""
    cut = lambda k, t: t[a // 128:-(-b // 128)] if "scale" in k else t[a:b]
    return {k: None if v is None else {j: cut(k, v[j])} for k, v in d.items()}


@pytest.mark.parametrize("pdt,master", [(F32, False), (BF16, False), (BF16, True)])
def test_long_items_of_ragged_lists(monkeypatch, pdt, master):
    say(f"[adamw-large] {pdt} master={master}")
    assert sum(SIZES) >= 2048 * 8192
    rng = np.random.default_rng(31)
    s = _lists(rng, SIZES, pdt, F32, 8, master)
    opt = B.make_adamw(**s)
    assert opt.list.item == 8192
    words = oadam.words
    n = SIZES[LARGE]
    last = n // 8192 * 8192
    # the first items' borders, passes of 2048 inside one, some far ones, the ragged end
    windows = [(0, 4096), (8064, 10368), (12288, 16512), (8192 * 1000 - 128, 8192 * 1001), (last - 256, n)]
    for t in (1, 2):
        keep = {k: None if v is None else [x.clone() for x in v] for k, v in s.items()}
        B.adamw(opt, lr=1e-3, step=t, seed=77, **HY)
        torch.cuda.synchronize()
        small = lambda d: {k: None if v is None else [v[j] if j != LARGE else v[j][:0] for j in range(len(SIZES))]
                           for k, v in d.items()}
        before = _snap(small(keep))
        for j, size in enumerate(SIZES):
            if j != LARGE:
                _check(before, s, j, t, 1e-3, 8, 77)
        for a, b in windows:
            monkeypatch.setattr(oadam, "words", lambda seed, t_, j, m, start=0: words(seed, t_, j, m, a))
            old, new = _part(keep, LARGE, a, b), _part(s, LARGE, a, b)
            old = {k: None if v is None else {LARGE: _np(v[LARGE])} for k, v in old.items()}
            _check(old, new, LARGE, t, 1e-3, 8, 77)
            monkeypatch.setattr(oadam, "words", words)
        # and no pass of an item was left out: every run of 2048 has parameters that moved.  (Not every one has to:
        # an update of about lr = 1e-3 is below half a bf16 step, 2^-9 of the value, of every p above 0.5.)
        moved = (s["p"][LARGE] != keep["p"][LARGE])[:n // 2048 * 2048].view(-1, 2048)
        assert bool(moved.any(1).all())
        assert bool((s["v"][LARGE].reshape(-1)[:n // 128 * 128].view(-1, 128) != 0).any(1).all())
