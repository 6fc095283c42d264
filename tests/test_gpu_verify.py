"""Verification of drafted tokens against whole-number arithmetic on the host:
every token and count must be equal."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import gather_lora_matmul_amd as L
from gpu_helpers import log

TD = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def fixed(x):
    x = np.where(np.isnan(x), 0.0, x).astype(np.float64)
    return np.floor(np.clip(x, 0.0, 1.0) * 2.0 ** 44).astype(np.int64)


def oracle(k, drafted, target, draft, u, us):
    """Rows as numpy float32; k drafted tokens of each sequence (-1: idle)."""
    tokens, counts = [], []
    a = r = 0
    V = target.shape[1]
    for s, n in enumerate(k):
        if n < 0:
            counts.append(0)
            continue
        done = 0
        while done < n:
            c = int(drafted[r + done])
            if not 0 <= c < V:
                break
            q = np.float32(1.0) if draft is None else draft[r + done, c]
            if not np.float32(u[r + done]) * q < target[a + done, c]:
                break
            done += 1
        p = target[a + done]
        with np.errstate(invalid="ignore"):
            if done == n:
                w = p
            elif draft is not None:
                w = p - draft[r + done]
            else:
                w = p.copy()
                if 0 <= drafted[r + done] < V:
                    w[drafted[r + done]] = 0
        w = fixed(w)
        if w.sum() == 0:
            w = fixed(p)
        total = int(w.sum())
        uu = min(max(float(us[s]), 0.0), 1 - 2.0 ** -24)
        level = total * int(np.floor(uu * 2 ** 31)) >> 31
        tok = int(np.searchsorted(np.cumsum(w), level, side="right")) if total else -1
        tokens += [int(x) for x in drafted[r:r + done]] + [tok] + [-1] * (n - done)
        counts.append(done + 1)
        a += n + 1
        r += n
    return np.array(tokens, np.int32), np.array(counts, np.int32)


def run(k, drafted, target, draft, u, us, stream=None):
    qs = torch.tensor(np.concatenate([[0], np.cumsum(np.array(k) + 1)]).astype(np.int32)).cuda()
    n = len(k)
    ws = torch.full((max(1, L.lora_spec_verify_workspace_size(n, target.shape[1])),), 0xFF, dtype=torch.uint8, device="cuda")
    tokens = torch.full((target.shape[0],), 77, dtype=torch.int32, device="cuda")
    n_out = torch.full((n,), 77, dtype=torch.int32, device="cuda")
    L.lora_spec_verify(qs, drafted, target, draft, u, us, tokens, n_out, ws, stream=stream)
    torch.cuda.synchronize()
    return tokens.cpu().numpy(), n_out.cpu().numpy()


def make(k, V, dtype, seed, ld=0, sharp=2.0, near=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, nd = sum(x + 1 for x in k), sum(x for x in k if x > 0)
    lt = torch.randn((n, V), device="cuda", generator=g) * sharp
    rows = [i for i in range(n)]
    keep, a = [], 0
    for x in k:
        keep += rows[a:a + max(x, 0)]
        a += x + 1
    ldr = lt[torch.tensor(keep, dtype=torch.int64, device="cuda")] + near * torch.randn((nd, V), device="cuda", generator=g)
    t = torch.zeros((n, V + ld), device="cuda", dtype=TD[dtype])
    d = torch.zeros((nd, V + ld), device="cuda", dtype=TD[dtype])
    t[:, :V] = torch.softmax(lt, -1).to(TD[dtype])
    d[:, :V] = torch.softmax(ldr, -1).to(TD[dtype])
    t, d = t[:, :V], d[:, :V]
    drafted = torch.multinomial(d.float() + 1e-30, 1, generator=g)[:, 0].to(torch.int32) if nd else \
        torch.zeros(0, dtype=torch.int32, device="cuda")
    u = torch.rand(nd, device="cuda", generator=g)
    us = torch.rand(len(k), device="cuda", generator=g)
    return drafted, t, d, u, us


def compare(k, drafted, t, d, u, us):
    got = run(k, drafted, t, d, u, us)
    want = oracle(k, drafted.cpu().numpy(), t.float().cpu().numpy(), None if d is None else d.float().cpu().numpy(),
                  u.cpu().numpy(), us.cpu().numpy())
    assert np.array_equal(got[1], want[1]), (got[1], want[1])
    assert np.array_equal(got[0], want[0]), np.argwhere(got[0] != want[0])[:5]
    return got


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 1000, 2048, 2049, 32000, 50257])
def test_random_drafts(dtype, V):
    k = [0, 4, 1, -1, 7, 3, 0, -1, 2, 5]
    for seed in range(3):
        log("[case] verify %s V %d seed %d" % (dtype, V, seed))
        compare(k, *make(k, V, dtype, seed, ld=(0, 3, 8)[seed], sharp=(2.0, 0.3, 4.0)[seed]))


def test_largest_vocabulary_and_many_drafts():
    k = [70, 0, 130]
    compare(k, *make(k, 1 << 18, "f32", 5, near=0.05))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_drafts_without_probabilities(dtype):
    k = [3, 0, 5, 1]
    drafted, t, d, u, us = make(k, 777, dtype, 6, sharp=0.2)
    top = t.float().argmax(1).to(torch.int32)
    drafted[0] = top[0]
    u[0] = 0.0
    compare(k, drafted, t, None, u, us)


def test_everything_and_nothing_accepted():
    k = [4, 4]
    drafted, t, d, u, us = make(k, 500, "f32", 7)
    same = torch.cat([t[0:4], t[5:9]])
    got = compare(k, drafted, t, same.contiguous(), u * 0.999, us)   # the draft is the target
    assert list(got[1]) == [5, 5]
    got = compare(k, drafted, t, d, u * 0 + 1.0, us)                 # a number of one refuses unless p > q
    far = torch.zeros_like(d)
    far[:, 3] = 1.0
    drafted[:] = 3
    t2 = t.clone()
    t2[:, 3] = 0
    got = compare(k, drafted, t2, far, u, us)
    assert list(got[1]) == [1, 1]


def test_residual_of_zero_and_rows_of_nothing():
    # the draft above the target everywhere: the target's own probabilities; all zero, NaN and infinite rows
    k = [1, 1, 0, 0, 1]
    V = 300
    g = torch.Generator(device="cuda").manual_seed(8)
    t = torch.softmax(torch.randn((8, V), device="cuda", generator=g), -1)
    d = t[[0, 2, 6]] * 2
    drafted = torch.tensor([5, 6, 400], dtype=torch.int32, device="cuda")   # the last is no token
    t[4] = 0
    t[5, :] = float("nan")
    t[5, 17] = float("inf")
    t[5, 19] = -1.0
    u = torch.full((3,), 0.9, device="cuda")
    us = torch.tensor([0.0, 0.999999, 0.5, 0.5, 0.3], device="cuda")
    got = compare(k, drafted, t, d, u, us)
    assert got[0][4] == -1 and got[0][5] == 17


def test_levels_at_the_boundaries():
    # weights that are exact powers of two and numbers at the edges of their intervals
    V = 4096
    t = torch.zeros((6, V), device="cuda")
    t[:, 100] = 0.25
    t[:, 2047] = 0.25
    t[:, 2048] = 0.25
    t[:, 4095] = 0.25
    us = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.24999999, 1.0], device="cuda")
    e = torch.zeros(0, device="cuda")
    got = compare([0] * 6, e.to(torch.int32), t, None, e, us)
    assert list(got[0]) == [100, 2047, 2048, 4095, 100, 4095]


def test_graph_replays():
    k = [2, 0, 4]
    drafted, t, d, u, us = make(k, 5000, "f32", 9)
    qs = torch.tensor([0, 3, 4, 9], dtype=torch.int32).cuda()
    ws = torch.empty(L.lora_spec_verify_workspace_size(3, 5000), dtype=torch.uint8, device="cuda")
    tokens = torch.empty(9, dtype=torch.int32, device="cuda")
    n_out = torch.empty(3, dtype=torch.int32, device="cuda")
    call = L.prepare_spec_verify(qs, drafted, t, d, u, us, tokens, n_out, ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(torch.cuda.current_stream())
    gen = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(4):
        u.copy_(torch.rand(6, device="cuda", generator=gen))
        us.copy_(torch.rand(3, device="cuda", generator=gen))
        tokens.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        want = oracle(k, drafted.cpu().numpy(), t.cpu().numpy(), d.cpu().numpy(), u.cpu().numpy(), us.cpu().numpy())
        assert np.array_equal(tokens.cpu().numpy(), want[0]) and np.array_equal(n_out.cpu().numpy(), want[1])


def test_rows_that_share_memory_are_refused():
    # rows expanded from one would have no stride: the call must not read past them
    vocab, dev = 40, "cuda"
    i32 = dict(dtype=torch.int32, device=dev)
    row = torch.full((1, vocab), 1 / vocab, device=dev)
    ws = torch.empty(L.lora_spec_verify_workspace_size(2, vocab), dtype=torch.uint8, device=dev)
    args = lambda target, draft: (torch.tensor([0, 2, 4], **i32), torch.zeros(2, **i32), target, draft,
                                  torch.zeros(2, device=dev), torch.zeros(2, device=dev),
                                  torch.empty(4, **i32), torch.empty(2, **i32), ws)
    with pytest.raises(L.LoraError, match="target_ld"):
        L.lora_spec_verify(*args(row.expand(4, vocab), None))
    with pytest.raises(L.LoraError, match="draft_ld"):
        L.lora_spec_verify(*args(row.repeat(4, 1), row.expand(2, vocab)))
