"""Temperatures whose reciprocal is not finite in fp32 are refused by every call of
the operators on sampled tokens, on a host without a GPU."""
import pytest

from test_token_ops_abi import FAKE, FAR, N, V, lib  # noqa: F401


@pytest.mark.parametrize("T", [1e-45, 1e-40, 2.9e-39, 4e-39])
def test_temperatures_without_a_finite_reciprocal(lib, T):  # noqa: F811
    import ctypes

    from logits_sampling_gb300._token_ops import _Policy, _Preference
    rows = [FAKE, 1, V, V, N, FAKE]
    policy = ctypes.byref(_Policy(0x10000, 0x10000, 0x10000, None, 0.2, 0.2, 0.0, 0.1, 2, 0.0, 0))
    preference = ctypes.byref(_Preference(0x10000, 2, None, None, 0, 0.1, 0.0, 0.0, 0))
    assert lib.ls_token_log_probs(*rows, T, FAR, None, FAR, None, None) == 1
    assert lib.ls_token_log_probs_backward(*rows, T, FAKE, None, None, FAR, V, None) == 1
    assert lib.ls_policy_loss(*rows, policy, T, FAR, FAR, FAR, None, None) == 1
    assert lib.ls_policy_loss_backward(*rows, T, FAKE, None, FAR, V, None) == 1
    assert lib.ls_policy_loss_grad(*rows, policy, T, FAKE, FAR, FAR, V, None, None) == 1
    assert lib.ls_preference_loss(*rows, preference, T, FAR, None, FAR, None, None) == 1
    assert lib.ls_preference_loss_backward(*rows, T, FAKE, 2, None, FAR, V, None) == 1
