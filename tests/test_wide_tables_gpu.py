"""Tables far wider than the batch's contexts, as a call that is captured for the longest one has them: the forms are
chosen by the width, the results are those of the lengths."""
import numpy as np
import pytest
import torch

import test_sparse_gpu
import test_tree_gpu

pytestmark = pytest.mark.gpu

WIDE = 8192


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_attention_25_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def widen(bt):
    return np.pad(bt, ((0, 0), (0, WIDE - bt.shape[1])), constant_values=-1)


TREES = [[(210, 7)], [(0, 1)], [(400, 33), (30, 5), (0, 0), (17, 64)],
         [(int(p), int(n)) for p, n in np.random.default_rng(1).integers([0, 1], [900, 28], (30, 2))]]


@pytest.mark.parametrize("form", [0, 1, 2], ids=["chosen", "rows", "tiles"])
@pytest.mark.parametrize("reqs", TREES, ids=["one_user", "one_token", "ragged", "batch"])
@pytest.mark.parametrize("hq,hkv,d,dtype", [(8, 2, 64, "bf16"), (16, 2, 128, "fp8_e4m3")])
def test_trees(form, reqs, hq, hkv, d, dtype, monkeypatch):
    monkeypatch.setattr(test_tree_gpu.Case, "form", form, raising=False)
    c = test_tree_gpu.Case(1, reqs, hq, hkv, d, dtype)
    c.bt = widen(c.bt)
    c.run_check()


@pytest.mark.parametrize("dtype", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("reqs", [[(3000, [2999])], [(40, [39, 20]), (700, [699]), (0, [])]], ids=["one_user", "ragged"])
def test_selection_and_lists(reqs, dtype):
    test_sparse_gpu.Case(2, reqs, 8, 2, 64, dtype, width=WIDE).whole(16, 1, 2)
    test_sparse_gpu.Case(3, reqs, 8, 2, 64, dtype, width=WIDE).whole(3000, 1, 2)      # lists far longer than the contexts
