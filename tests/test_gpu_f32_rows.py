"""float32 decode with more than 32 query rows per KV head whose key range is
split between CTAs: the merge of the split pieces covers every row (up to 64
rows of a pass, 2048 four-column items at D = 128)."""
import numpy as np
import pytest
import torch

import parity_util as pu
from paged_kv_cache_182_gb300 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,H,KV,NQ", [(128, 5, 1, 7), (128, 8, 2, 16), (64, 16, 1, 4), (128, 33, 1, 2)])
def test_every_row_of_a_split_segment_is_written(D, H, KV, NQ):
    spec = W.Spec("f32_rows", "f32", B=2, H=H, KV=KV, D=D, BLOCK=16, NQ=NQ, causal=True)
    w = W.make(spec, seed=D + H, lens=[1500, 260])
    dev = w.to("cuda")
    from paged_kv_cache_182_gb300 import binding

    out = torch.full((2, H, NQ, D), float("nan"), device="cuda")
    binding.decode(*dev.tensors(), scale=spec.scale, causal=True, out=out)
    torch.cuda.synchronize()
    want = pu.run_oracle(w)
    assert np.all(np.isfinite(out.cpu().numpy()))
    pu.check(out, want, "f32", "f32", "rows past 32")
