"""The alignment operators refuse what their kernels cannot take, before
anything is launched (CPU only): the torch functions by exceptions, the C
entry points by status codes."""
import ctypes

import pytest
import torch

import linear_cross_entropy_tiled_amd as flce

S, L = 4, 6


def _tokens(**change):
    a = dict(logps=torch.zeros(S, L), ref_logps=torch.zeros(S, L), mask=torch.ones(S, L, dtype=torch.bool),
             offsets=None)
    a.update(change)
    return a


PACKED = dict(logps=torch.zeros(20), ref_logps=torch.zeros(20), mask=None, offsets=torch.zeros(S + 1, dtype=torch.int64))


@pytest.mark.parametrize("change,opts,exc", [
    ({}, {}, ValueError),                                                         # consistent, but on the CPU
    (PACKED, {}, ValueError),
    (dict(logps=torch.zeros(S, L, dtype=torch.float64)), {}, TypeError),
    (dict(ref_logps=torch.zeros(S, L, dtype=torch.bfloat16)), {}, TypeError),
    (dict(mask=torch.ones(S, L)), {}, TypeError),
    (dict(mask=torch.ones(S, L - 1, dtype=torch.bool)), {}, ValueError),
    (dict(ref_logps=torch.zeros(S, L + 1)), {}, ValueError),
    (dict(logps=torch.zeros(L, S).t()), {}, ValueError),                          # columns, not rows
    (dict(logps=torch.zeros(1, L).expand(S, L)), {}, ValueError),                 # overlapping rows
    (dict(logps=torch.zeros(S * L)), {}, ValueError),                             # packed without offsets
    (dict(logps=torch.zeros(3, L), ref_logps=None, mask=None), {}, ValueError),   # an odd number of answers
    (dict(ref_logps=torch.zeros(S, L, requires_grad=True)), {}, ValueError),
    ({**PACKED, "offsets": torch.zeros(S + 1)}, {}, TypeError),
    ({**PACKED, "offsets": torch.zeros(0, dtype=torch.int64)}, {}, ValueError),
    ({**PACKED, "offsets": torch.zeros(2 * S + 2, dtype=torch.int64)[::2]}, {}, ValueError),
    ({**PACKED, "logps": torch.zeros(4, 5)}, {}, ValueError),
    ({}, dict(beta=0.0), ValueError),
    ({}, dict(beta=float("nan")), ValueError),
    ({}, dict(loss_type="exp"), ValueError),
    ({}, dict(label_smoothing=1.5), ValueError),
    ({}, dict(loss_type="hinge", label_smoothing=0.1), ValueError),
    ({}, dict(margin=float("inf")), ValueError),
    ({}, dict(reduction="sequence_mean"), ValueError),
])
def test_preference_loss_rejects(change, opts, exc):
    with pytest.raises(exc):
        flce.preference_loss(**_tokens(**change), **opts)


def _policy(**change):
    a = dict(logps=torch.zeros(S, L), old_logps=torch.zeros(S, L), advantages=torch.zeros(S))
    a.update(change)
    return a


@pytest.mark.parametrize("change,exc", [
    ({}, ValueError),
    (dict(old_logps=torch.zeros(S, L, dtype=torch.float16)), TypeError),
    (dict(advantages=torch.zeros(S, dtype=torch.float64)), TypeError),
    (dict(advantages=torch.zeros(S + 1)), ValueError),
    (dict(advantages=torch.zeros(1, S)), ValueError),
    (dict(advantages=torch.zeros(2 * S)[::2]), ValueError),
    (dict(advantages=torch.zeros(S, requires_grad=True)), ValueError),
    (dict(old_logps=torch.zeros(S, L, requires_grad=True)), ValueError),
    (dict(entropy=torch.zeros(S, L + 2)), ValueError),
    (dict(kl_coef=0.1), ValueError),
    (dict(entropy_coef=0.1), ValueError),
    (dict(clip_low=-0.1), ValueError),
    (dict(clip_high=float("nan")), ValueError),
    (dict(dual_clip=1.0), ValueError),
    (dict(kl_coef=float("inf"), ref_logps=torch.zeros(S, L)), ValueError),
    (dict(reduction="token"), ValueError),
    # packed, as many tokens as sequences: per token or per sequence?
    (dict(logps=torch.zeros(S), old_logps=torch.zeros(S), offsets=torch.zeros(S + 1, dtype=torch.int32)), ValueError),
    (dict(advantages_per_sequence=False), ValueError),
    (dict(advantages=torch.zeros(S, L), advantages_per_sequence=True), ValueError),
])
def test_policy_loss_rejects(change, exc):
    with pytest.raises(exc):
        flce.policy_loss(**_policy(**change))


def _view(p=None, ld=0):
    return flce.flce_token_view(p, ld)


NONE = _view()


def _pp(**change):
    a = dict(n_seqs=S, length=L, dtype=1, reduction=2, type=0, flags=0, length_normalize=0, reserved=0, beta=0.1,
             label_smoothing=0.0, margin=0.0)
    a.update(change)
    return flce.flce_preference_params(**a)


@pytest.mark.parametrize("change,code", [
    (dict(n_seqs=3), flce.FLCE_ERR_INVALID_ARG), (dict(n_seqs=-2), flce.FLCE_ERR_INVALID_ARG),
    (dict(length=-1), flce.FLCE_ERR_INVALID_ARG), (dict(dtype=3), flce.FLCE_ERR_INVALID_ARG),
    (dict(reduction=3), flce.FLCE_ERR_INVALID_ARG), (dict(type=3), flce.FLCE_ERR_INVALID_ARG),
    (dict(flags=2), flce.FLCE_ERR_INVALID_ARG), (dict(length_normalize=2), flce.FLCE_ERR_INVALID_ARG),
    (dict(reserved=1), flce.FLCE_ERR_INVALID_ARG), (dict(beta=0.0), flce.FLCE_ERR_INVALID_ARG),
    (dict(label_smoothing=2.0), flce.FLCE_ERR_INVALID_ARG),
    (dict(type=1, label_smoothing=0.1), flce.FLCE_ERR_INVALID_ARG),
    (dict(margin=float("nan")), flce.FLCE_ERR_INVALID_ARG),
    (dict(n_seqs=1 << 25), flce.FLCE_ERR_UNSUPPORTED), (dict(length=1 << 41), flce.FLCE_ERR_UNSUPPORTED),
    (dict(n_seqs=1 << 20, length=1 << 21), flce.FLCE_ERR_UNSUPPORTED),
])
def test_preference_abi_codes(change, code):
    p = _pp(**change)
    with pytest.raises(flce.FlceError) as e:
        flce.flce_preference_workspace_size(p)
    assert e.value.code == code
    assert flce.flce_preference_forward(p, _view(16), NONE, NONE, None, 16, 16, 16, 16, 1 << 30, None) == code
    if change.get("n_seqs", 0) < 1 << 20 and change.get("length", 0) < 1 << 41:
        assert flce.flce_preference_backward(p, 16, 16, NONE, None, 16, None) == code


def test_preference_abi_pointers_and_workspace():
    p = _pp()
    need = flce.flce_preference_workspace_size(p)
    ok = dict(logps=_view(256), ref=NONE, mask=NONE, offsets=None, loss=16, rewards=16, seq=16, ws=256, nbytes=need)

    def call(**change):
        a = {**ok, **change}
        return flce.flce_preference_forward(p, a["logps"], a["ref"], a["mask"], a["offsets"], a["loss"], a["rewards"],
                                            a["seq"], a["ws"], a["nbytes"], None)

    bad, odd = flce.FLCE_ERR_INVALID_ARG, flce.FLCE_ERR_UNSUPPORTED
    for name in ("loss", "rewards", "seq", "ws"):
        assert call(**{name: None}) == bad, name
    assert call(logps=NONE) == bad
    assert call(logps=_view(256, L - 1)) == bad          # rows would overlap
    assert call(mask=_view(256, 2)) == bad
    assert call(logps=_view(257)) == odd                 # not aligned to an element
    assert call(loss=18) == odd and call(ws=264) == odd and call(offsets=260) == odd
    assert call(nbytes=need - 1) == flce.FLCE_ERR_WORKSPACE_TOO_SMALL
    assert flce.flce_preference_backward(p, None, 16, NONE, None, 16, None) == bad
    assert flce.flce_preference_backward(p, 16, None, NONE, None, 16, None) == bad
    assert flce.flce_preference_backward(p, 16, 16, NONE, None, None, None) == bad
    assert flce.flce_preference_backward(p, 16, 16, NONE, None, 17, None) == odd


def _lp(**change):
    a = dict(n_seqs=S, length=L, dtype=0, reduction=2, flags=0, reserved=0, clip_low=0.2, clip_high=0.2, dual_clip=0.0,
             kl_coef=0.0, entropy_coef=0.0)
    a.update(change)
    return flce.flce_policy_params(**a)


@pytest.mark.parametrize("change", [
    dict(n_seqs=-1), dict(length=-1), dict(dtype=4), dict(reduction=4), dict(flags=4), dict(reserved=1),
    dict(clip_low=-1.0), dict(clip_high=float("nan")), dict(dual_clip=0.5), dict(dual_clip=float("inf")),
    dict(kl_coef=float("nan")), dict(entropy_coef=float("inf"))])
def test_policy_abi_codes(change):
    p = _lp(**change)
    with pytest.raises(flce.FlceError) as e:
        flce.flce_policy_workspace_size(p)
    assert e.value.code == flce.FLCE_ERR_INVALID_ARG
    assert flce.flce_policy_backward(p, 16, 16, 16, NONE, None, 16, 16, None) == flce.FLCE_ERR_INVALID_ARG


def test_policy_abi_pointers_and_workspace():
    def call(p=None, **change):
        p = p or _lp()
        need = flce.flce_policy_workspace_size(p)
        a = dict(logps=_view(256), old=_view(256), ref=NONE, ent=NONE, adv=_view(256), mask=NONE, offsets=None, loss=16,
                 unit=16, weights=16, metrics=None, ws=256, nbytes=need)
        a.update(change)
        if a["nbytes"] == "short":
            a["nbytes"] = need - 1
        return flce.flce_policy_forward(p, a["logps"], a["old"], a["ref"], a["ent"], a["adv"], a["mask"], a["offsets"],
                                        a["loss"], a["unit"], a["weights"], a["metrics"], a["ws"], a["nbytes"], None)

    bad, odd = flce.FLCE_ERR_INVALID_ARG, flce.FLCE_ERR_UNSUPPORTED
    for name in ("loss", "weights", "ws"):
        assert call(**{name: None}) == bad, name
    for name in ("logps", "old", "adv"):
        assert call(**{name: NONE}) == bad, name
    assert call(_lp(flags=2), adv=NONE) == bad
    assert call(_lp(kl_coef=0.1)) == bad and call(_lp(entropy_coef=0.1)) == bad
    assert call(old=_view(256, 3)) == bad
    assert call(unit=20) == odd and call(metrics=20) == odd and call(old=_view(258)) == odd
    assert call(nbytes="short") == flce.FLCE_ERR_WORKSPACE_TOO_SMALL
    assert flce.flce_policy_backward(_lp(), 16, None, 16, NONE, None, 16, None, None) == bad
    assert flce.flce_policy_backward(_lp(), 16, 16, None, NONE, None, 16, None, None) == bad
    assert flce.flce_policy_backward(_lp(), None, 16, 16, NONE, None, 16, None, None) == bad


def test_workspace_counts_one_partial_sum_per_chunk_and_sequence():
    # 16 bytes for each (chunk, sequence) pair that can meet: chunks of 256 tokens up to 8192 x 256 tokens
    assert flce.flce_preference_workspace_size(_pp(n_seqs=2, length=256)) == 256
    assert flce.flce_preference_workspace_size(_pp(n_seqs=1000, length=512)) == (2000 * 16 + 255) // 256 * 256
    p = _pp(n_seqs=0, length=0)
    assert flce.flce_preference_workspace_size(p) >= 16
    assert ctypes.sizeof(flce.flce_preference_params) == 64 and ctypes.sizeof(flce.flce_policy_params) == 72
