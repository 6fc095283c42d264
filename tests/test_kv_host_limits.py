"""Host-side checks at the limits of the KV calls' arguments (no GPU; see test_kv_host for the host-only pools)."""
import ctypes

import pytest

import gather_lora_matmul_amd as L
from test_kv_host import ARG, STATE, attend_status, batch, host_pool, kv, ref


@pytest.fixture
def pool():
    h = host_pool()
    yield h
    L.lora_pool_destroy(h)


@pytest.mark.parametrize("heads", [8, 64])
def test_tokens_are_not_left_out_for_a_longest_length_of_none(pool, heads):
    # the call goes on to its work (here: to the host-only refusal), with the workspace of a length of one
    size = {}
    for max_q in (0, 1):
        n = ctypes.c_size_t()
        assert L.lib().lora_kv_attend_workspace_size(pool, ref(kv()), ref(batch(max_q=max_q)), heads, ref(n)) == 0
        size[max_q] = n.value
        args = dict(heads=heads, q_ld=heads * 128, out_ld=heads * 128)
        assert attend_status(pool, kv(), batch(max_q=max_q), ws_bytes=n.value, **args) == STATE
        assert attend_status(pool, kv(), batch(max_q=max_q), ws_bytes=n.value - 1, **args) == ARG
    assert size[0] == size[1]
