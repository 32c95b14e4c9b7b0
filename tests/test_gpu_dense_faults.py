"""Dense attention on the GPU: inputs that were once answered wrongly, in both kernels."""
import numpy as np
import pytest

import workloads as wlm
from dense_cases import DenseCase, check_attention
from oracle import dsa_oracle as o

pytestmark = pytest.mark.gpu


def put(a):
    import torch
    return torch.from_numpy(np.array(a)).cuda()


def attend(case, tensors=None, longest=None, check=True, scale=128 ** -0.5, **mods):
    """(out as float64, lse as float64) with rows that no kernel wrote at -7."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    cache, batch, q = tensors or case.gpu()
    out = torch.full((case.rows, case.heads, 128), -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.rows, case.heads), -7.0, dtype=torch.float32, device="cuda")
    mods = {k: put(v) if isinstance(v, np.ndarray) else v for k, v in mods.items()}
    dsa.paged_attention(cache, batch, q, scale, max_query_len=longest or max(1, int(case.q_lens.max())), out=out, lse=lse,
                        check=check, **mods)
    torch.cuda.synchronize()
    return o.bf16_to_f64(wlm.torch_to_bits(out)), lse.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("B,stride", [(64, 40), (4096, 8192)])
def test_starts_that_run_back_are_refused(B, stride):
    """Every other request names the same 2,048 rows of 16 heads: 128 groups of 256 pairs each time.  With 2,048 of them and
    8,192 tiles of 128 keys a group, the sum of the tiles would be 2^31."""
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    rows, P = 2048, 128
    starts = np.zeros(B + 1, np.int32)
    starts[1::2] = rows
    cache = dsa.BlockKvCache(4, P, 1)
    table = torch.zeros((B, stride), dtype=torch.int32, device="cuda")
    lens = torch.full((B,), stride * P, dtype=torch.int32, device="cuda")
    batch = dsa.Batch(table, lens, put(starts), num_rows=rows, max_seq_len=stride * P)
    q = torch.zeros((rows, 16, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.full((rows, 16, 128), -7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(dsa.DsaError, match="BAD_LENGTH"):
        dsa.paged_attention(cache, batch, q, max_query_len=rows, out=out, check=True)
    assert torch.all(out == -7.0).item()


@pytest.mark.parametrize("group", [1, 5, 6, 20, 24])
def test_equal_calls_give_equal_bits_whatever_ran_between_them(group):
    """Columns of a tile that no query fills keep what an earlier call left in shared memory: they do not count."""
    case = DenseCase(37, [2300, 1800, 2777, 900] * 10, [1] * 40, 64, 2, group)
    wide = 8 if group <= 8 else 32
    others = [DenseCase(38, [2500] * 40, [1] * 40, 64, 2, wide), DenseCase(39, [700] * 40, [1] * 40, 64, 2, wide)]
    for c, up in zip(others, (64.0, 2.0 ** -20)):
        c.q_bits = wlm.bf16_bits((c.q * up).astype(np.float32))
    tensors, busy = case.gpu(), [c.gpu() for c in others]
    first = None
    for between in (None, 0, 1, 0, None):
        if between is not None:
            attend(others[between], busy[between])
        got = attend(case, tensors)
        first = first or got
        same = np.array_equal(got[0], first[0]) and np.array_equal(got[1], first[1])
        assert same, f"after {between}"
    check_attention(*first, case.oracle())
