"""The Python binding of the attention block's calls, without a GPU."""
import types

import numpy as np
import pytest

import expert_routing_grouped_gb300 as moe


@pytest.mark.parametrize("off,n_seq,T,want", [(None, None, 7, 7), ([0, 3, 7], None, 7, 2), ([0, 3, 7], 1, 7, 1),
                                              ([0, 7], None, 7, 1), (None, 7, 7, 7)])
def test_sequences_of_a_batch(monkeypatch, off, n_seq, T, want):
    """q_off says how many sequences there are where n_seq does not: T of them would read
    offsets, lengths and pages past their arrays' ends."""
    seen = {}

    def call(name, at):
        def f(*args):
            seen[name] = args[at]
            return moe.MOE_OK
        return f
    monkeypatch.setattr(moe, "lib", types.SimpleNamespace(moe_kv4_append=call("append", 7),
                                                          moe_kv4_attention=call("attention", 6)))
    monkeypatch.setattr(moe, "_stream", lambda stream: None)
    x = np.zeros(16, np.float32)
    q_off = None if off is None else np.array(off, np.int32)
    moe.kv4_append(x, x, x, x, x, T, 1, 64, 16, 1, 1, q_off=q_off, n_seq=n_seq)
    moe.kv4_attention(x, x, x, x, T, 1, 1, 64, 16, 1, 1, x, None, q_off=q_off, n_seq=n_seq)
    assert seen == {"append": want, "attention": want}
