"""Softmax attention against the 64-bit definition in every form that the plan
of a call can take; the plan is asserted, so that a change of its estimates
does not move these sizes to another form unseen."""
import pytest
import torch

import rank_latent_attention_flare_b200 as fl
from test_gpu_attn import BF, check, tensors

# name: (B, Hq, Hk, Nq, Nk, causal, q_lens, k_lens), (query tiles a CTA, heads a
# tile, keys split), (dK and dV split, dQ split, CTAs stay where D <= 64)
CASES = {
    # two query tiles a CTA, the last CTA's second one empty
    "pairs": ((2, 16, 4, 513, 700, False, [513, 257], [700, 333]), (2, 1, False),
              (False, False, False)),
    # ... with different numbers of key tiles, lengths that empty one or both
    "pairs_causal": ((4, 20, 20, 520, 520, True, [520, 100, 385, 256], [520, 100, 500, 40]),
                     (2, 1, False), (False, False, True)),
    "pairs_even": ((3, 50, 25, 256, 256, True, None, None), (2, 1, False), (False, False, True)),
    # ... fewer keys than queries: rows, and whole tiles, that see no key
    "pairs_few_keys": ((4, 40, 10, 300, 200, True, None, [200, 1, 129, 77]), (2, 1, False),
                       (False, False, False)),
    # ... a chunk of a sequence: every query sees more keys than there are queries
    "pairs_chunk": ((3, 20, 20, 257, 1500, True, None, [1500, 1281, 300]), (2, 1, False),
                    (False, False, True)),
    # ... and the keys split, in the forward and for dQ
    "pairs_split": ((2, 4, 2, 130, 9000, True, [130, 129], [9000, 6000]), (2, 1, True),
                    (False, True, True)),
    "one_tile": ((2, 10, 10, 200, 300, True, None, [300, 201]), (1, 1, False),
                 (False, False, True)),
    "one_tile_split": ((1, 2, 1, 200, 2000, False, None, None), (1, 1, True),
                       (False, True, True)),
    "heads_in_a_tile": ((2, 8, 2, 20, 100, True, None, [100, 60]), (1, 4, False),
                        (False, False, True)),
    "heads_in_a_tile_split": ((2, 8, 2, 5, 3500, True, [5, 2], [3500, 1]), (1, 4, True),
                              (False, True, True)),
    "dkv_split": ((1, 4, 1, 3000, 200, False, None, None), (1, 1, False), (True, False, True)),
}


def plan(name, D):
    (B, Hq, Hk, Nq, Nk, causal, _, _), fwd, bwd = CASES[name]
    qt, hpt, splits = fl.attn_plan(False, B, Hq, Hk, Nq, Nk, D, BF, causal)
    dkv, dq, stay = fl.attn_plan(True, B, Hq, Hk, Nq, Nk, D, BF, causal)
    return (qt, hpt, splits > 1), (dkv > 1, dq > 1, bool(stay)), (*fwd, *bwd[:2],
                                                                  bwd[2] and D <= 64)


@pytest.mark.parametrize("D", [16, 32, 64, 80, 96, 128])
@pytest.mark.parametrize("name", CASES)
def test_plans(name, D):
    """On a B200, or on the host for one."""
    fwd, bwd, want = plan(name, D)
    assert (*fwd, *bwd) == want


def test_plan_refuses_what_the_calls_refuse():
    for bad in (dict(B=0), dict(Hq=5), dict(D=12), dict(D=136)):
        args = {**dict(B=1, Hq=4, Hk=2, Nq=10, Nk=10, D=64), **bad}
        with pytest.raises(fl.FlareError):
            fl.attn_plan(False, *args.values(), BF)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [16, 32, 64, 80, 96, 128])
@pytest.mark.parametrize("name", CASES)
def test_against_definition(name, D):
    fwd, bwd, want = plan(name, D)
    assert (*fwd, *bwd) == want
    B, Hq, Hk, Nq, Nk, causal, q_lens, k_lens = CASES[name][0]
    check(*tensors(BF, B, Hq, Hk, Nq, Nk, D, seed=40, layout="bnhd" if D % 64 else "bhnd"), causal,
          q_lens, k_lens)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [8, 56, 104, 120])
def test_padded_heads(D):
    """Head sizes that the kernels fill up with zeros, in pairs of query tiles."""
    check(*tensors(BF, 2, 16, 4, 513, 300, D, seed=41), True, [513, 300], None)


@pytest.mark.gpu
def test_pairs_repeat_and_match_single_tiles():
    """A row's result does not depend on the tile it shares a CTA with: the first
    queries of a call that takes pairs, alone, give the same bits (all of their
    keys are visible, whole and in the same tiles)."""
    q, k, v, _ = tensors(BF, 3, 50, 25, 256, 384, 64, seed=42)
    assert all(fl.attn_plan(False, 3, 50, 25, n, 384, 64, BF)[0] == 2 for n in (256, 512))
    y = fl.attn_fwd(q, k, v)
    for _ in range(3):
        assert torch.equal(y, fl.attn_fwd(q, k, v))
    more = torch.cat((q, q.flip(2)), 2)   # the pairs keep their place, others follow
    assert torch.equal(fl.attn_fwd(more, k, v)[:, :, :256], y)
