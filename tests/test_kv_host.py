"""Host-side checks of the KV cache and of the verification of drafts (no GPU):
geometry, workspace sizes and what the entry points refuse.  Calls on host-only
pools report a wrong argument first and LORA_E_STATE when nothing else is wrong,
so every refusal shows before anything could be launched; the pointers below are
never read."""
import ctypes

import pytest

import gather_lora_matmul_amd as L

ARG, STATE, UNSUPPORTED = -1, -5, -7
P = 0x7F0000001000  # aligned, never read


def host_pool(page=4096, dtype="bf16", n_pages=64, act=None):
    return L.lora_pool_create(page, L.DTYPE_CODE[dtype], n_pages, 1, 8, [(64, 64)], flags=L.LORA_POOL_HOST_ONLY,
                              act_dtype=None if act is None else L.DTYPE_CODE[act])


@pytest.fixture
def pool():
    h = host_pool()
    yield h
    L.lora_pool_destroy(h)


@pytest.mark.parametrize("page,pool_dt,act,heads,D,kv,T", [
    (4096, "bf16", "bf16", 8, 128, "bf16", 32),     # 8192 bytes: 32 rows of 256
    (4096, "f16", "f16", 1, 64, "f16", 64),
    (4096, "bf16", "bf16", 256, 128, "e4m3", 64),   # one byte an element
    (1000, "bf16", "bf16", 3, 128, "bf16", 0),      # 2000 bytes: 7 rows, rounded down to 0
    (1104, "bf16", "bf16", 3, 128, "bf16", 8),      # 2208 bytes: 8 rows and a tail
    (1104, "bf16", "bf16", 3, 64, "bf16", 16),      # 17 rows, rounded down to 16
    (5008, "e4m3", "f16", 2, 128, "f16", 16),       # FP8 pool, 16-bit cache: 19 rows
    (5008, "e4m3", "f16", 2, 128, "e4m3", 32),      # 39 rows, rounded down to 32
])
def test_layout(page, pool_dt, act, heads, D, kv, T):
    h = host_pool(page, pool_dt, 64, act)
    try:
        if T == 0:
            with pytest.raises(L.LoraError):
                L.lora_kv_layout(h, heads, D, L.DTYPE_CODE[kv])
        else:
            scales = 64 * T if kv == "e4m3" else 0
            assert L.lora_kv_layout(h, heads, D, L.DTYPE_CODE[kv]) == (T, 2 * heads, scales)
    finally:
        L.lora_pool_destroy(h)


def kv(heads=2, D=128, dtype=None, scales=None):
    return L.KvDesc(heads, D, L.LORA_BF16 if dtype is None else dtype, scales)


def batch(n_seqs=2, n_tokens=10, max_q=8, max_blocks=4, q_start=P, kv_len=P, table=P):
    return L.KvBatchDesc(n_seqs, n_tokens, max_q, max_blocks, q_start, kv_len, table)


def ref(x):
    return None if x is None else ctypes.byref(x)


def status(st):
    if st:
        assert L.lib().lora_last_error()
    return st


BAD_CACHES = [(None, ARG), (kv(heads=0), ARG), (kv(heads=257), ARG), (kv(D=96), UNSUPPORTED), (kv(D=256), UNSUPPORTED),
              (kv(dtype=L.LORA_F16), ARG), (kv(dtype=L.LORA_F32), ARG), (kv(dtype=77), ARG)]
# scales are looked at where they are read: not by lora_kv_layout or the workspace's size
BAD_SCALES = [(kv(dtype=L.LORA_FP8_E4M3), ARG), (kv(dtype=L.LORA_FP8_E4M3, scales=P + 8), ARG)]
BAD_SIZES = [None, batch(n_seqs=-1), batch(n_seqs=1025), batch(n_tokens=-1), batch(n_tokens=(1 << 24) + 1),
             batch(max_q=-1), batch(max_q=11), batch(max_blocks=0), batch(max_blocks=(1 << 23) + 1)]
BAD_POINTERS = [batch(q_start=None), batch(kv_len=None), batch(table=None), batch(q_start=P + 2),
                batch(kv_len=P + 1), batch(table=P + 2)]


def copy_status(pool, d, b, k=P, v=P, ld=256):
    w = status(L.lib().lora_kv_write(pool, ref(d), ref(b), k, v, ld, None))
    assert w == status(L.lib().lora_kv_read(pool, ref(d), ref(b), k, v, ld, None))
    return w


def attend_status(pool, d, b, q=P, q_ld=1024, heads=8, scale=0.1, window=0, out=P, out_ld=1024, lse=None, ws=P,
                  ws_bytes=1 << 30):
    return status(L.lib().lora_kv_attend(pool, ref(d), ref(b), q, q_ld, heads, scale, window, out, out_ld, lse, ws,
                                         ws_bytes, None))


def size_status(pool, d, b, heads=8, out=True):
    n = ctypes.c_size_t()
    return status(L.lib().lora_kv_attend_workspace_size(pool, ref(d), ref(b), heads, ref(n) if out else None))


def test_valid_calls_reach_the_host_only_check(pool):
    # the yardstick of the refusals below: the same calls with nothing wrong
    assert copy_status(pool, kv(), batch()) == STATE
    assert attend_status(pool, kv(), batch()) == STATE
    assert copy_status(pool, kv(dtype=L.LORA_FP8_E4M3, scales=P), batch()) == STATE
    assert size_status(pool, kv(), batch()) == 0
    # nothing to do: nothing is read, not even the rows' pointers
    for b in (batch(n_seqs=0, q_start=None, kv_len=None, table=None), batch(n_tokens=0, max_q=0)):
        assert copy_status(pool, kv(), b, k=None, v=None, ld=0) == 0
        assert attend_status(pool, kv(), b, q=None, out=None, ws=None, ws_bytes=0) == 0


@pytest.mark.parametrize("i", range(len(BAD_CACHES)))
def test_bad_caches(pool, i):
    d, want = BAD_CACHES[i]
    assert status(L.lib().lora_kv_layout(pool, ref(d), None, None, None)) == want
    assert copy_status(pool, d, batch()) == want
    assert attend_status(pool, d, batch()) == want
    assert size_status(pool, d, batch()) == want


@pytest.mark.parametrize("i", range(len(BAD_SCALES)))
def test_bad_scales(pool, i):
    d, want = BAD_SCALES[i]
    assert status(L.lib().lora_kv_layout(pool, ref(d), None, None, None)) == 0
    assert copy_status(pool, d, batch()) == want and attend_status(pool, d, batch()) == want


@pytest.mark.parametrize("i", range(len(BAD_SIZES) + len(BAD_POINTERS)))
def test_bad_batches(pool, i):
    b = (BAD_SIZES + BAD_POINTERS)[i]
    assert copy_status(pool, kv(), b) == ARG
    assert attend_status(pool, kv(), b) == ARG
    assert size_status(pool, kv(), b) == (ARG if i < len(BAD_SIZES) else 0)


def test_bad_pools():
    assert copy_status(None, kv(), batch()) == ARG and attend_status(None, kv(), batch()) == ARG
    assert size_status(None, kv(), batch()) == ARG
    h = host_pool(dtype="f32")
    assert copy_status(h, kv(), batch()) == UNSUPPORTED and attend_status(h, kv(), batch()) == UNSUPPORTED
    L.lora_pool_destroy(h)


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 2), dict(ld=248),
                                dict(ld=260), dict(ld=0), dict(ld=-256)])
def test_bad_rows(pool, kw):
    assert copy_status(pool, kv(), batch(), **kw) == ARG


@pytest.mark.parametrize("kw,want", [
    (dict(heads=1), ARG), (dict(heads=3), ARG), (dict(heads=0), ARG), (dict(heads=-2), ARG),
    (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG),
    (dict(scale=float("inf")), ARG), (dict(scale=3e38), ARG), (dict(window=-1), ARG),
    (dict(q=None), ARG), (dict(q=P + 8), ARG), (dict(q_ld=1016), ARG), (dict(q_ld=1028), ARG),
    (dict(out=None), ARG), (dict(out=P + 4), ARG), (dict(out_ld=0), ARG), (dict(lse=P + 2), ARG),
    (dict(ws=None), ARG), (dict(ws_bytes=0), ARG), (dict(ws=P + 128), ARG),
])
def test_bad_attend(pool, kw, want):
    assert attend_status(pool, kv(), batch(), **kw) == want


def test_too_much_work_is_refused(pool):
    # 2^24 tokens of 64 query heads on one kv head: more than 2^28 query rows of it
    b = batch(n_tokens=1 << 24, max_q=1 << 24)
    assert attend_status(pool, kv(heads=1), b, heads=64, q_ld=8192, out_ld=8192) == UNSUPPORTED
    assert size_status(pool, kv(heads=1), b, heads=64) == UNSUPPORTED
    # 1024 sequences of 2^28 positions of 256 heads: more units than the cut counts
    b = batch(n_seqs=1024, n_tokens=1 << 20, max_q=1 << 20, max_blocks=1 << 23)
    assert attend_status(pool, kv(heads=256), b, heads=256, q_ld=1 << 15, out_ld=1 << 15) == UNSUPPORTED


def test_workspace_is_what_the_size_call_says(pool):
    n = ctypes.c_size_t()
    for b in (batch(), batch(max_q=1), batch(n_seqs=1024, n_tokens=4096, max_q=4000), batch(n_seqs=0)):
        assert L.lib().lora_kv_attend_workspace_size(pool, ref(kv()), ref(b), 8, ref(n)) == 0
        assert 0 < n.value < 1 << 30
        if b.n_seqs:
            assert attend_status(pool, kv(), b, ws_bytes=n.value) == STATE
            assert attend_status(pool, kv(), b, ws_bytes=n.value - 1) == ARG
    assert size_status(pool, kv(), batch(), out=False) == ARG


def verify_desc(**kw):
    f = dict(n_seqs=3, n_tokens=9, n_drafts=6, vocab=1000, dtype=L.LORA_F32, target_ld=1000,
             draft_ld=1000, q_start_dev=P, drafted_dev=P, target_dev=P, draft_dev=P, u_accept_dev=P, u_sample_dev=P,
             tokens_dev=P, n_out_dev=P)
    f.update(kw)
    d = L.VerifyDesc()
    for k, v in f.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("kw", [
    dict(n_seqs=-1), dict(n_seqs=65536), dict(vocab=0), dict(vocab=(1 << 18) + 1), dict(n_tokens=-1),
    dict(n_drafts=-1), dict(n_drafts=10), dict(dtype=L.LORA_FP8_E4M3), dict(dtype=9), dict(target_ld=999),
    dict(draft_ld=999), dict(target_ld=0), dict(target_ld=-1000),
    dict(q_start_dev=None), dict(drafted_dev=None), dict(target_dev=None), dict(u_accept_dev=None),
    dict(u_sample_dev=None), dict(tokens_dev=None), dict(n_out_dev=None),
    dict(q_start_dev=P + 2), dict(drafted_dev=P + 1), dict(target_dev=P + 2), dict(draft_dev=P + 2),
    dict(u_accept_dev=P + 2), dict(u_sample_dev=P + 3), dict(tokens_dev=P + 1), dict(n_out_dev=P + 2),
    dict(dtype=L.LORA_BF16, target_dev=P + 1), dict(dtype=L.LORA_F16, draft_dev=P + 1),
])
def test_bad_verify(kw):
    assert status(L.lib().lora_spec_verify(ref(verify_desc(**kw)), P, 1 << 30, None)) == ARG


def test_bad_verify_workspace():
    d = verify_desc()
    n = ctypes.c_size_t()
    assert L.lib().lora_spec_verify_workspace_size(3, 1000, ref(n)) == 0 and n.value > 0
    assert status(L.lib().lora_spec_verify(ref(d), None, n.value, None)) == ARG
    assert status(L.lib().lora_spec_verify(ref(d), P, n.value - 1, None)) == ARG
    assert status(L.lib().lora_spec_verify(ref(d), P + 8, n.value, None)) == ARG
    assert status(L.lib().lora_spec_verify(None, P, n.value, None)) == ARG
    assert status(L.lib().lora_spec_verify_workspace_size(3, 1000, None)) == ARG
    assert status(L.lib().lora_spec_verify_workspace_size(3, 0, ref(n))) == ARG
    # no sequences: nothing is read
    assert status(L.lib().lora_spec_verify(ref(verify_desc(n_seqs=0, q_start_dev=None)), None, 0, None)) == 0


def test_binding_refuses_what_the_kernels_would_misread(pool):
    torch = pytest.importorskip("torch")
    cache = L.KvCache(pool, 2, 128, L.LORA_BF16)
    i32 = dict(dtype=torch.int32)
    with pytest.raises(TypeError, match="int32"):
        L.KvBatch(torch.zeros(3, dtype=torch.int64), torch.zeros(2, **i32), torch.zeros(2, 2, 2, 4, **i32), 10, 8)
    with pytest.raises(ValueError, match="q_start"):
        L.KvBatch(torch.zeros(2, **i32), torch.zeros(2, **i32), torch.zeros(2, 2, 2, 4, **i32), 10, 8)
    for shape in ((2, 2, 2), (3, 2, 2, 4), (2, 1, 2, 4)):
        with pytest.raises(ValueError, match="table"):
            L.KvBatch(torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(*shape, **i32), 10, 8)
    with pytest.raises(ValueError, match="device tensor"):
        L.KvBatch(torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(2, 2, 2, 4, **i32), 10, 8)
    with pytest.raises((TypeError, ValueError), match="scales"):
        L.KvCache(pool, 2, 128, L.LORA_FP8_E4M3)
    with pytest.raises(TypeError, match="scales"):
        L.KvCache(pool, 2, 128, L.LORA_FP8_E4M3, scales=torch.zeros(1 << 16, dtype=torch.int8))
    with pytest.raises(ValueError, match="scales"):
        L.KvCache(pool, 2, 128, L.LORA_FP8_E4M3, scales=torch.zeros(8, dtype=torch.uint8))

    class Batch:  # rows are checked against the call's tokens and the table's heads
        desc = batch()
        table = torch.zeros(2, 2, 2, 4, **i32)

    class Wide(Batch):
        table = torch.zeros(2, 2, 3, 4, **i32)

    rows = torch.zeros(10, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="k: dtype"):
        L.prepare_kv_write(cache, Batch, rows.half(), rows)
    for bad in (rows[:9], rows.view(10, 256), rows.view(10, 4, 64), torch.zeros(10, 3, 128, dtype=torch.bfloat16)):
        with pytest.raises(ValueError, match="k: "):
            L.prepare_kv_write(cache, Batch, bad, rows)
    with pytest.raises(ValueError, match="heads"):
        L.prepare_kv_read(cache, Wide, rows, rows)
    with pytest.raises(ValueError, match="device tensor"):
        L.prepare_kv_read(cache, Batch, rows, rows)
