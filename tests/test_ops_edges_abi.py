"""Sizes at the ends of the dense operators' ranges, without a GPU."""
import expert_routing_grouped_gb300 as moe

INT_MAX = 2 ** 31 - 1


def test_balance_workspace_is_zero_for_refused_sizes():
    """T * top_k is at most 2^26 whatever top_k, and n_seq at most 65535."""
    ws = moe.balance_workspace
    for T in ((1 << 26) + 1, 1 << 27, INT_MAX - 455, INT_MAX - 30, INT_MAX):
        assert ws(T, 8, 1) == 0
    assert ws(1 << 26, 8, 1) > 0 and ws(4, 8, 65535) > 0
    assert ws(4, 8, 65536) == 0 and ws(4, 8, INT_MAX) == 0
    assert ws(-1, 8, 1) == 0 and ws(4, -1, 1) == 0 and ws(4, 8, -1) == 0


def test_linear_wait_limit_refuses():
    assert moe.lib.moe_linear_wait_limit(-1) == moe.MOE_ERR_ARG
    assert moe.lib.moe_linear_wait_limit(2000000) == moe.MOE_OK


def test_linear_status_refuses():
    assert moe.lib.moe_linear_status(None) == moe.MOE_ERR_ARG


def test_balance_of_no_tokens_refuses():
    """The outputs that T = 0 sets to zero are checked like any call's."""
    a = [(i + 1) << 26 for i in range(4)]   # loss, counts, tokens, prob

    def call(loss, counts, tokens, prob):
        return moe.lib.moe_balance_loss(None, None, None, None, a[0] << 4, 0, 16, 2, 3, 0, 0, 0.01, None,
                                        0, loss, counts, tokens, prob, None, 0, None, 0, None)

    assert call(a[0] + 2, a[1], a[2], a[3]) == moe.MOE_ERR_ARG
    assert call(a[0], a[1], a[1] + 64, a[3]) == moe.MOE_ERR_ARG
    assert call(a[0], a[1], a[2], None) == moe.MOE_OK
