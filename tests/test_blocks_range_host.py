"""Host checks beside test_blocks_host: results of a wrong kind are refused by name, and the low end of the gates' gradient in
float64 agrees with differences. No GPU work."""
import os

import numpy as np
import pytest
import torch

import blocks_ref as ref

moe = pytest.importorskip("bit_quantized_moe_topk_amd")
if not os.path.exists(moe.LIB_PATH):
    pytest.skip("libmoe.so not built (run __graft_entry__.build())", allow_module_level=True)


@pytest.mark.parametrize("out", [object(), torch.zeros(4, 256), (torch.zeros(4, 256),)])
def test_results_of_a_wrong_kind(out):
    x, w = torch.zeros(4, 256), torch.ones(256)
    for call in (lambda: moe.fp8_quantize(x, out=out), lambda: moe.rms_norm(x, w, out=out),
                 lambda: moe.rms_norm(x, w, fp8=True, out=moe.Norm(None, x, out))):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("level", [-95.0, -300.0, 12.0])
def test_gradient_form_at_the_ends(level):
    """Renormalised sigmoid gates against central differences, where scores are far from 1/2."""
    rng = np.random.default_rng(int(abs(level)))
    x = level + rng.standard_normal((3, 7))
    idx, _ = ref.route(x, 3, None, "sigmoid", 1, 1, 2, True, 1.5)
    d = rng.standard_normal((3, 3))

    def gates(x):
        q = np.take_along_axis(ref.scores(x, "sigmoid"), idx.astype(np.int64), 1)
        return 1.5 * q / q.sum(1, keepdims=True)
    got, _ = ref.route_gradient(x, idx, d, "sigmoid", True, 1.5)
    for e in range(7):
        h = np.zeros_like(x)
        h[:, e] = 1e-4
        diff = ((gates(x + h) - gates(x - h)) * d).sum(1) / 2e-4
        assert np.allclose(got[:, e], diff, atol=1e-8)
