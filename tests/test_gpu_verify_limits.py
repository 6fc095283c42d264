"""Verification of drafted tokens where the counts do not agree."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import gather_lora_matmul_amd as L


@pytest.mark.parametrize("vocab", [50, 40000])   # one launch and two
def test_rows_of_drafts_that_are_not_there_hold_no_old_tokens(vocab):
    # three sequences of 3, 4 and 2 drafted tokens, of which the call has 4: the second one's pass its end
    g = torch.Generator(device="cuda").manual_seed(1)
    i32 = dict(dtype=torch.int32, device="cuda")
    target = torch.softmax(torch.randn((12, vocab), device="cuda", generator=g), -1)
    drafted = target[:4].argmax(1).to(torch.int32)
    tokens, n_out = torch.full((12,), 77, **i32), torch.full((3,), 77, **i32)
    ws = torch.empty(L.lora_spec_verify_workspace_size(3, vocab), dtype=torch.uint8, device="cuda")
    u = torch.zeros(4, device="cuda")
    L.lora_spec_verify(torch.tensor([0, 4, 9, 12], **i32), drafted, target, None, u, torch.full((3,), 0.5, device="cuda"),
                       tokens, n_out, ws)
    torch.cuda.synchronize()
    t, n = tokens.cpu().numpy(), n_out.cpu().numpy()
    # the first is whole (numbers of 0 accept), the others draw one token of their first row
    assert n.tolist() == [4, 1, 1] and t[:3].tolist() == drafted[:3].tolist()
    w = np.floor(target[[3, 4, 9]].double().cpu().numpy() * 2.0 ** 44).astype(np.int64)
    for at, row in zip((3, 4, 9), w):
        assert t[at] == np.searchsorted(np.cumsum(row), int(row.sum()) >> 1, side="right")
    assert np.all(t[5:9] == -1) and np.all(t[10:] == -1)
