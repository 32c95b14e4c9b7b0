"""Dense attention over the 8-bit K/V cache on the GPU against the float64 oracle."""
import numpy as np
import pytest

import workloads as wlm
from dense_cases import DenseCase, check_attention
from oracle import dsa_oracle as o

pytestmark = pytest.mark.gpu


def run(case, scale=128 ** -0.5, max_query_len=None, fill=None, **mods):
    import torch
    import deepseek_sparse_mla_gb300 as dsa
    cache, batch, q = case.gpu()
    out = torch.full((case.rows, case.heads, 128), -7.0 if fill is None else fill, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.rows, case.heads), -7.0, dtype=torch.float32, device="cuda")
    dev = {k: torch.from_numpy(np.array(v)).cuda() if isinstance(v, np.ndarray) else v for k, v in mods.items()}
    if "prefix" in dev:
        dev["prefix_lens"] = dev.pop("prefix")
    dsa.paged_attention(cache, batch, q, scale, max_query_len=max_query_len or max(1, int(case.q_lens.max())), out=out, lse=lse,
                        check=True, **dev)
    torch.cuda.synchronize()
    return o.bf16_to_f64(wlm.torch_to_bits(out)), lse.cpu().numpy().astype(np.float64)


def reach(case, mods):
    return float(case.slopes.max()) * 64.0 if "slopes" in mods else 0.0


CASES = [
    # seq_lens, q_lens, page, kv heads, group
    ([1], [1], 16, 1, 1),
    ([300], [1], 64, 2, 8),
    ([127, 128, 129], [1, 1, 1], 16, 2, 4),
    ([0, 1, 0, 257], [1, 1, 0, 1], 32, 1, 8),
    ([640, 5, 1000, 33], [1, 1, 1, 1], 128, 2, 5),
    ([513, 260], [4, 4], 64, 2, 8),
    ([700, 90, 41], [3, 1, 4], 16, 1, 3),
    ([700, 90, 41, 200], [2, 0, 5, 1], 32, 2, 16),
    ([400], [1], 64, 1, 64),
    ([300, 17, 64], [37, 17, 1], 32, 2, 6),
    ([1300], [150], 64, 1, 8),
    ([260, 129], [260, 129], 128, 1, 12),
]


@pytest.mark.parametrize("n", range(len(CASES)))
def test_matches_the_oracle(n):
    seq, new, P, kv, group = CASES[n]
    case = DenseCase(100 + n, seq, new, P, kv, group)
    got, lse = run(case)
    check_attention(got, lse, case.oracle())


@pytest.mark.parametrize("n", [2, 5, 9, 10])
@pytest.mark.parametrize("which", ["cap", "slopes", "prefix", "all"])
def test_capped_scores_distance_bias_and_prefix(n, which):
    seq, new, P, kv, group = CASES[n]
    case = DenseCase(200 + n, seq, new, P, kv, group)
    mods = {}
    if which in ("cap", "all"):
        mods["softcap"] = 2.5
    if which in ("slopes", "all"):
        mods["slopes"] = case.slopes
    if which in ("prefix", "all"):
        mods["prefix"] = np.array([min(L, 45 + 100 * i) for i, L in enumerate(seq)], np.int32)
    got, lse = run(case, **mods)
    check_attention(got, lse, case.oracle(**mods), softcap=mods.get("softcap", 0.0), reach=reach(case, mods))
