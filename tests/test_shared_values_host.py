"""The bound of the outputs of decode behind shared prefixes, on the CPU: over marked values every
mistake in the products of weights and V breaks it, for each row and head."""
import pytest
import torch

import shared_ref as S
import values_ref as V

MISTAKES = ["nothing", "tile left out", "tile taken twice", "V of the next tile", "page left out",
            "V of another page"]


@pytest.mark.parametrize("kind", ["bf16", "e4m3_tensor", "e4m3_token", "int8_tensor", "int8_token"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_mistakes_break_the_bound(kind, dim):
    w = V.mark(S.make([(250, [(40, 2), (90, 1)])], kind=kind, dim=dim, hkv=2, group=2, seed=dim))
    for stage1 in (False, True):
        o, bound, _, _ = V.attention(w, [4000, 4000], stage1)
        assert bool((bound < 0.03 + o.abs() / 20).all())
        for what in MISTAKES:
            for at in (0, 1300, 3850):
                wrong = (V.mistaken(w, what, at) - o).abs() > bound
                assert bool(wrong.any(-1).all()), (what, at, stage1)


def test_the_marked_values_are_the_caches():
    for kind in ("bf16", "e4m3_tensor", "e4m3_token", "int8_token"):
        w = V.mark(S.make([(20, [(40, 2)])], kind=kind, seed=1))
        c, s = w.cache[1], w.scale[1]
        x = c.view(S.E4M3).double() if "e4m3" in kind else c.double()
        if s is not None:
            x = x * (s.double() if s.dim() == 1 else s.double()[..., None])
        used = V.used_pages(w)
        assert torch.equal(x[used], w.values[1][used])
