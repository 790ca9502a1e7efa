"""The example of a decoder layer's attention: prompts, then graph-replayed steps."""
import os
import sys

import numpy as np
import pytest

import kv_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))


@pytest.mark.parametrize("bits", [4, 8])
def test_prompts_then_steps(bits):
    """The layer's attention equals the definition over the quantized tokens: its output
    projection is the same call in both, so the attention's tolerance passes through the
    weights, plus what one code of the activation's quantization is worth."""
    import attention_block as ex
    import w4a8_int8_quantized_gb300 as w8
    blk, outs, qkvs = ex.run(prompts=(150, 20, 1), steps=5, bits=bits)
    h, kvh, d = blk.heads, blk.kv_heads, blk.head_dim
    codes, scale = (t.cpu().numpy().astype(np.float64) for t in blk.w_out)
    weight = codes * scale.reshape(-1, 1)
    at = [0] * len(qkvs)
    for b in range(len(qkvs[0])):
        seq = torch.cat([step[b] for step in qkvs]).cpu().numpy()
        q, k, v = np.split(seq, [h, h + kvh], 1)
        kc, ks = ref.quantize(k, bits)
        vc, vs = ref.quantize(v, bits)
        o, _, tol, _ = ref.attend(q, kc, ks, vc, vs, d ** -0.5)
        o, tol = o.reshape(len(seq), -1), tol.reshape(len(seq), -1)
        want = o @ weight.T
        # quantization of the activation: half a code each, and the attention's own error
        half = np.abs(o).max(1, keepdims=True) / 254
        slack = (tol + half * 1.01) @ np.abs(weight).T + 2.0 ** -10 * np.abs(want) + 2.0 ** -24
        row = 0
        for i, step in enumerate(qkvs):
            n = len(step[b])
            got = outs[i][at[i]:at[i] + n].double().cpu().numpy()
            assert (np.abs(got - want[row:row + n]) <= slack[row:row + n]).all()
            # far below that bound on the whole: rounding errors are independent
            err = got - want[row:row + n]
            assert np.linalg.norm(err) <= 0.05 * np.linalg.norm(want[row:row + n])
            at[i] += n
            row += n
    assert w8.w8a8_check_status() == 0
