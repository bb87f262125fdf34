"""Which tokens and which of a teacher's slots the vocabulary head's losses count,
against the formulas in 64 bits."""
import math

import pytest
import torch

import mixture_experts_layer_permute_amd as M

from _gpu import banner, needs_gpu
from _head import check, inputs, reference

pytestmark = [pytest.mark.gpu, needs_gpu]


@pytest.mark.parametrize("T", [64, 700])
def test_a_token_whose_slots_score_minus_infinity_is_left_out(T):
    """Its row of x is not read (NaN here), as for a label outside the vocabulary; few
    tokens and many slots look at the slots in kernels of their own."""
    d, V, K = 64, 300, 40
    banner("head slots of -infinity", T)
    x, Wv, labels, weight, (idx, score, tw) = inputs(T, d, V, K=K, seed=T)
    score[::5] = -math.inf
    labels[::10] = -1
    teacher = (idx, score, tw)
    for lab, w, gone in ((labels, weight, slice(0, None, 10)), (None, None, slice(0, None, 5))):
        ref = reference(x, Wv, lab, w, teacher, 1.5)
        dirty = x.clone()
        dirty[gone] = float("nan")
        for limit in (0, 1):
            res = M.moe_head_distill_grad(dirty, Wv, teacher, 1.5, lab, w, limit=limit)
            check(res, ref)
            assert bool((res["dx"][gone] == 0).all()) and bool((res["kd"][gone] == 0).all())
        check(M.moe_head_distill(dirty, Wv, teacher[:2], 1.5, lab), ref)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 100, 256])
def test_the_loss_alone_of_few_tokens_passes_over_nan_rows(T, dt):
    """Up to 256 tokens every row is scored, those without a label too: nothing of
    them reaches another row."""
    d, V = 192, 701
    banner("head NaN rows", T, dt)
    x, Wv, labels, _, _ = inputs(T, d, V, dt, seed=T)
    labels[::3] = -1
    want = reference(x, Wv, labels, dt=dt)
    x[::3] = float("nan")
    check(M.moe_head_xent(x, Wv, labels), want)


@pytest.mark.parametrize("K", [1, 70])
def test_a_teachers_nan_shows(K):
    """In the token that has it, whether its other slots have scores or not, and in
    no other's kd and row of dx."""
    T, d, V = 90, 64, 200
    banner("head teacher NaN", K)
    x, Wv, labels, weight, (idx, score, tw) = inputs(T, d, V, K=K, seed=K)
    idx.clamp_(min=0)
    want = reference(x, Wv, labels, weight, (idx, score, tw), 2.0)
    bad = torch.tensor([4, 40, 77])
    score[4] = float("nan")
    score[40, K - 1] = float("nan")
    score[77] = -math.inf
    score[77, 0] = float("nan")
    res = M.moe_head_distill_grad(x, Wv, (idx, score, tw), 2.0, labels, weight)
    assert bool(res["kd"][bad].isnan().all()) and bool(res["dx"][bad].isnan().any(1).all())
    ok = torch.ones(T, dtype=torch.bool)
    ok[bad] = False
    check({"kd": res["kd"][ok], "dx": res["dx"][ok]},
          {n: tuple(t[ok.cuda()] for t in want[n]) for n in ("kd", "dx")})
    check({"loss": res["loss"], "lse": res["lse"]}, want)
