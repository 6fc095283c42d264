"""Host-side checks of trees of drafted tokens and of eviction (no GPU): what the entry points and the binding
refuse.  As in the checks of the cache's other calls, a host-only pool reports a wrong argument first and
LORA_E_STATE when nothing else is wrong; the pointers below are never read."""
import ctypes

import pytest

import gather_lora_matmul_amd as L
from test_kv_host import ARG, BAD_CACHES, BAD_POINTERS, BAD_SCALES, BAD_SIZES, P, STATE, UNSUPPORTED, batch, host_pool, kv, ref, status


@pytest.fixture
def pool():
    h = host_pool()
    yield h
    L.lora_pool_destroy(h)


def tree(words=1, seen=P, depth=P):
    return L.KvTreeDesc(words, 0, seen, depth)


def build_status(n_seqs=2, n_tokens=10, q_start=P, parent=P, words=1, window=0, seen=P, depth=P):
    return status(L.lib().lora_kv_tree_build(n_seqs, n_tokens, q_start, parent, words, window, seen, depth, None))


def attend_status(pool, d, b, t=tree(), q=P, q_ld=1024, heads=8, scale=0.1, window=0, out=P, out_ld=1024, lse=None,
                  ws=P, ws_bytes=1 << 30):
    return status(L.lib().lora_kv_attend_tree(pool, ref(d), ref(b), ref(t), q, q_ld, heads, scale, window, out, out_ld,
                                              lse, ws, ws_bytes, None))


def weigh_status(pool, d, b, q=P, q_ld=1024, heads=8, scale=0.1, window=0, lse=P, decay=1.0, before=None, weights=P,
                 w_ld=100, ws=P, ws_bytes=1 << 30):
    return status(L.lib().lora_kv_weigh(pool, ref(d), ref(b), q, q_ld, heads, scale, window, lse, decay, before, weights,
                                        w_ld, ws, ws_bytes, None))


def select_status(pool, d, b, weights=P, w_ld=100, budget=8, sinks=2, recent=3, keep=P, keep_ld=8, n_keep=P, ws=P,
                  ws_bytes=1 << 30):
    return status(L.lib().lora_kv_select(pool, ref(d), ref(b), weights, w_ld, budget, sinks, recent, keep, keep_ld,
                                         n_keep, ws, ws_bytes, None))


def compact_status(pool, d, b, keep=P, heads=1, keep_ld=8, n_keep=P, from_new=0, weights=None, w_ld=0):
    return status(L.lib().lora_kv_compact(pool, ref(d), ref(b), keep, heads, keep_ld, n_keep, from_new, weights, w_ld,
                                          None))


CALLS = [attend_status, weigh_status, select_status, compact_status]


def test_valid_calls_reach_the_host_only_check(pool):
    for call in CALLS:
        assert call(pool, kv(), batch()) == STATE
        assert call(pool, kv(dtype=L.LORA_FP8_E4M3, scales=P), batch()) == STATE
        # nothing to do
        assert call(pool, kv(), batch(n_seqs=0, q_start=None, kv_len=None, table=None)) == 0
    empty = batch(n_tokens=0, max_q=0)
    assert attend_status(pool, kv(), empty, q=None, out=None, ws=None, ws_bytes=0) == 0
    # cached tokens fade without new ones, too
    assert weigh_status(pool, kv(), empty, q=None, lse=None) == STATE
    assert select_status(pool, kv(), empty) == STATE and compact_status(pool, kv(), empty) == STATE
    assert select_status(pool, kv(), batch(), budget=0, sinks=0, recent=0, keep=None, keep_ld=0) == STATE
    assert compact_status(pool, kv(), batch(), keep=None, keep_ld=0, n_keep=None) == 0
    assert compact_status(pool, kv(), batch(), heads=2, weights=P, w_ld=7, from_new=1) == STATE
    assert attend_status(pool, kv(), batch(), t=tree(16, depth=None)) == STATE
    assert attend_status(pool, kv(), batch(), window=5) == STATE
    assert build_status(n_seqs=0, q_start=None, parent=None, seen=None, depth=None) == 0
    assert build_status(n_tokens=0, q_start=None, parent=None, seen=None, depth=None) == 0


@pytest.mark.parametrize("call", CALLS)
def test_bad_caches_batches_and_pools(pool, call):
    for d, want in BAD_CACHES + BAD_SCALES:
        assert call(pool, d, batch()) == want
    for b in BAD_SIZES + BAD_POINTERS:
        assert call(pool, kv(), b) == ARG
    assert call(None, kv(), batch()) == ARG
    h = host_pool(dtype="f32")
    assert call(h, kv(), batch()) == UNSUPPORTED
    L.lora_pool_destroy(h)


@pytest.mark.parametrize("kw", [
    dict(n_seqs=-1), dict(n_seqs=1025), dict(n_tokens=-1), dict(n_tokens=(1 << 24) + 1), dict(words=0), dict(words=17),
    dict(words=-1), dict(window=-1), dict(q_start=None), dict(parent=None), dict(seen=None), dict(depth=None),
    dict(q_start=P + 2), dict(parent=P + 1), dict(seen=P + 4), dict(depth=P + 2)])
def test_bad_builds(kw):
    assert build_status(**kw) == ARG


@pytest.mark.parametrize("kw,want", [
    (dict(t=None), ARG), (dict(t=tree(0)), ARG), (dict(t=tree(17)), ARG), (dict(t=tree(seen=None)), ARG),
    (dict(t=tree(seen=P + 4)), ARG), (dict(t=tree(depth=P + 2)), ARG), (dict(t=tree(depth=None), window=3), ARG),
    (dict(heads=3), ARG), (dict(scale=0.0), ARG), (dict(scale=float("inf")), ARG), (dict(window=-1), ARG),
    (dict(q=None), ARG), (dict(q=P + 8), ARG), (dict(q_ld=1016), ARG), (dict(out=None), ARG), (dict(out_ld=1020), ARG),
    (dict(lse=P + 2), ARG), (dict(ws=None), ARG), (dict(ws_bytes=0), ARG), (dict(ws=P + 128), ARG)])
def test_bad_attention_of_trees(pool, kw, want):
    assert attend_status(pool, kv(), batch(), **kw) == want


@pytest.mark.parametrize("kw", [
    dict(heads=3), dict(heads=0), dict(scale=-1.0), dict(scale=float("nan")), dict(window=-1), dict(q=None),
    dict(q=P + 8), dict(q_ld=1000), dict(lse=None), dict(lse=P + 1), dict(decay=-0.1), dict(decay=1.5),
    dict(decay=float("nan")), dict(before=P + 2), dict(weights=None), dict(weights=P + 2), dict(w_ld=0), dict(w_ld=-4),
    dict(w_ld=(1 << 28) + 1)])
def test_bad_weighing(pool, kw):
    assert weigh_status(pool, kv(), batch(), **kw) == ARG


@pytest.mark.parametrize("kw", [
    dict(weights=None), dict(weights=P + 1), dict(w_ld=0), dict(budget=-1), dict(sinks=-1), dict(recent=-1),
    dict(sinks=4, recent=5), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(keep=None), dict(keep=P + 2), dict(keep_ld=7), dict(n_keep=None), dict(n_keep=P + 1),
    dict(ws=None), dict(ws_bytes=0), dict(ws=P + 64)])
def test_bad_selections(pool, kw):
    assert select_status(pool, kv(), batch(), **kw) == ARG


@pytest.mark.parametrize("kw", [
    dict(keep=None), dict(keep=P + 2), dict(heads=0), dict(heads=3), dict(heads=-1), dict(keep_ld=-1), dict(n_keep=None),
    dict(n_keep=P + 2), dict(weights=P + 1, w_ld=5), dict(weights=P, w_ld=0)])
def test_bad_compactions(pool, kw):
    assert compact_status(pool, kv(), batch(), **kw) == ARG


def test_workspaces_are_what_the_size_calls_say(pool):
    n = ctypes.c_size_t()
    for b in (batch(), batch(max_q=1), batch(n_seqs=1024, n_tokens=4096, max_q=4000), batch(n_tokens=0, max_q=0)):
        assert L.lib().lora_kv_select_workspace_size(pool, ref(kv()), ref(b), ref(n)) == 0 and n.value > 0
        assert select_status(pool, kv(), b, ws_bytes=n.value) == STATE
        assert select_status(pool, kv(), b, ws_bytes=n.value - 1) == ARG
        assert L.lib().lora_kv_weigh_workspace_size(pool, ref(kv()), ref(b), 8, ref(n)) == 0
        assert weigh_status(pool, kv(), b, ws=P if n.value else None, ws_bytes=n.value) == STATE
        if n.value:
            assert weigh_status(pool, kv(), b, ws_bytes=n.value - 1) == ARG
            assert weigh_status(pool, kv(), b, ws=P + 64) == ARG
    for d, b, want in [(kv(), BAD_SIZES[1], ARG), (kv(heads=0), batch(), ARG), (kv(D=96), batch(), UNSUPPORTED)]:
        assert status(L.lib().lora_kv_select_workspace_size(pool, ref(d), ref(b), ref(n))) == want
        assert status(L.lib().lora_kv_weigh_workspace_size(pool, ref(d), ref(b), 8, ref(n))) == want
    assert status(L.lib().lora_kv_select_workspace_size(pool, ref(kv()), ref(batch()), None)) == ARG
    assert status(L.lib().lora_kv_weigh_workspace_size(pool, ref(kv()), ref(batch()), 8, None)) == ARG
    assert status(L.lib().lora_kv_weigh_workspace_size(pool, ref(kv()), ref(batch()), 3, ref(n))) == ARG


def test_too_much_work_is_refused(pool):
    b = batch(n_seqs=1024, n_tokens=1 << 20, max_q=1 << 20, max_blocks=1 << 23)
    assert weigh_status(pool, kv(heads=256), b, heads=256, q_ld=1 << 15) == UNSUPPORTED
    assert attend_status(pool, kv(heads=256), b, heads=256, q_ld=1 << 15, out_ld=1 << 15) == UNSUPPORTED
    assert weigh_status(pool, kv(heads=1), batch(n_tokens=1 << 24, max_q=1 << 24), heads=64, q_ld=8192) == UNSUPPORTED


def verify_desc(**kw):
    f = dict(n_seqs=3, n_tokens=9, vocab=1000, dtype=L.LORA_F32, path_ld=4, target_ld=1000, q_start_dev=P, parent_dev=P,
             drafted_dev=P, target_dev=P, u_accept_dev=P, u_sample_dev=P, tokens_dev=P, path_dev=P, n_out_dev=P)
    f.update(kw)
    d = L.TreeVerifyDesc()
    for k, v in f.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw", [
    dict(n_seqs=-1), dict(n_seqs=65536), dict(vocab=0), dict(vocab=(1 << 18) + 1), dict(n_tokens=-1),
    dict(dtype=L.LORA_FP8_E4M3), dict(dtype=9), dict(path_ld=0), dict(path_ld=-3), dict(target_ld=999),
    dict(q_start_dev=None), dict(parent_dev=None), dict(drafted_dev=None), dict(target_dev=None),
    dict(u_accept_dev=None), dict(u_sample_dev=None), dict(tokens_dev=None), dict(path_dev=None), dict(n_out_dev=None),
    dict(q_start_dev=P + 2), dict(parent_dev=P + 1), dict(drafted_dev=P + 1), dict(target_dev=P + 2),
    dict(u_accept_dev=P + 2), dict(u_sample_dev=P + 3), dict(tokens_dev=P + 1), dict(path_dev=P + 2),
    dict(n_out_dev=P + 2), dict(dtype=L.LORA_BF16, target_dev=P + 1)])
def test_bad_tree_verification(kw):
    assert status(L.lib().lora_spec_verify_tree(ref(verify_desc(**kw)), P, 1 << 30, None)) == ARG


def test_bad_tree_verification_workspace():
    d, n = verify_desc(), ctypes.c_size_t()
    assert L.lib().lora_spec_verify_tree_workspace_size(3, 1000, ref(n)) == 0 and n.value > 0
    assert status(L.lib().lora_spec_verify_tree(ref(d), None, n.value, None)) == ARG
    assert status(L.lib().lora_spec_verify_tree(ref(d), P, n.value - 1, None)) == ARG
    assert status(L.lib().lora_spec_verify_tree(ref(d), P + 8, n.value, None)) == ARG
    assert status(L.lib().lora_spec_verify_tree(None, P, n.value, None)) == ARG
    assert status(L.lib().lora_spec_verify_tree_workspace_size(3, 1000, None)) == ARG
    assert status(L.lib().lora_spec_verify_tree_workspace_size(3, 0, ref(n))) == ARG
    assert status(L.lib().lora_spec_verify_tree(ref(verify_desc(n_seqs=0, q_start_dev=None)), None, 0, None)) == 0


def test_binding_refuses_what_the_kernels_would_misread(pool):
    torch = pytest.importorskip("torch")
    i32, i64 = dict(dtype=torch.int32), dict(dtype=torch.int64)
    for bad in (torch.zeros(4, 1, **i32), torch.zeros(4, **i64), torch.zeros(4, 17, **i64), torch.zeros(4, 0, **i64)):
        with pytest.raises(TypeError, match="seen"):
            L.KvTree(bad)
    with pytest.raises(TypeError, match="depth"):
        L.KvTree(torch.zeros(4, 1, **i64), torch.zeros(4, **i64))
    with pytest.raises(ValueError, match="depth"):
        L.KvTree(torch.zeros(4, 1, **i64), torch.zeros(3, **i32))
    with pytest.raises(ValueError, match="device tensor"):
        L.KvTree(torch.zeros(4, 1, **i64))

    cache = L.KvCache(pool, 2, 128, L.LORA_BF16)

    class Batch:
        desc = batch()
        table = torch.zeros(2, 2, 2, 4, **i32)

    class Wide(Batch):
        table = torch.zeros(2, 2, 3, 4, **i32)

    class Tree:
        seen = torch.zeros(9, 1, **i64)

    rows, w = torch.zeros(10, 2, 128, dtype=torch.bfloat16), torch.zeros(2, 2, 50)
    keep, n_keep = torch.zeros(2, 2, 8, **i32), torch.zeros(2, **i32)
    with pytest.raises(ValueError, match="heads"):
        L.prepare_kv_attend_tree(cache, Wide, Tree, rows, rows, 0.1)
    with pytest.raises(ValueError, match="heads"):
        L.prepare_kv_weigh(cache, Wide, rows, torch.zeros(10, 2), w, 0.1)
    with pytest.raises(ValueError, match="heads"):
        L.prepare_kv_select(cache, Wide, w, 8, keep, n_keep)
    with pytest.raises(ValueError, match="heads"):
        L.prepare_kv_compact(cache, Wide, keep, n_keep)
    with pytest.raises(TypeError, match="q: dtype"):
        L.prepare_kv_weigh(cache, Batch, rows.half(), torch.zeros(10, 2), w, 0.1)
    for bad in (torch.zeros(2, 50), torch.zeros(3, 2, 50), torch.zeros(2, 3, 50)):
        with pytest.raises(ValueError, match="weights: shape"):
            L.prepare_kv_select(cache, Batch, bad, 8, keep, n_keep)
    with pytest.raises(TypeError, match="weights: dtype"):
        L.prepare_kv_select(cache, Batch, w.double(), 8, keep, n_keep)
    with pytest.raises(ValueError, match="device tensor"):
        L.prepare_kv_select(cache, Batch, w, 8, keep, n_keep)
    for bad in (torch.zeros(3, 2, 8, **i32), torch.zeros(8, **i32)):
        with pytest.raises(ValueError, match="keep: shape"):
            L.prepare_kv_compact(cache, Batch, bad, n_keep)
    with pytest.raises(TypeError, match="keep: dtype"):
        L.prepare_kv_compact(cache, Batch, keep.long(), n_keep)
    with pytest.raises(ValueError, match="n_keep"):
        L.prepare_kv_compact(cache, Batch, keep, n_keep[:1])
    with pytest.raises(ValueError, match="device tensor"):
        L.prepare_kv_tree_build(n_keep, torch.zeros(4, **i32), torch.zeros(4, 1, **i64), torch.zeros(4, **i32))
    with pytest.raises(ValueError, match="target"):
        L.prepare_spec_verify_tree(n_keep, keep, keep, torch.zeros(4, 9), w, w, keep, keep, n_keep, None)
    with pytest.raises(TypeError, match="target"):
        L.prepare_spec_verify_tree(n_keep, keep, keep, torch.zeros(4, 9).double(), w, w, keep, keep, n_keep, None)
