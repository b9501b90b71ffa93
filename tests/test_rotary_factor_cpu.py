"""YaRN's factor on cosine and sine: 0.1 ln scale + 1 for longer contexts than the trained
one, 1 for no longer ones, where that would shrink (or, from e^-10 on, flip) every vector."""
import math

import pytest

import bit_block_quantized_nibble_amd as qbn


@pytest.mark.parametrize("scale", [1e-5, 0.5, 1.0, 1.0 + 2.0 ** -52, 1.5, 40.0])
def test_yarn_factor(scale):
    f, factor = qbn.rope_frequencies(64, scaling="yarn", scale=scale, original=4096)
    assert factor == (0.1 * math.log(scale) + 1 if scale > 1 else 1.0) and factor >= 1
    assert qbn.Rope.make(64, scaling="yarn", scale=scale, original=4096, device="cpu").factor == factor
    plain, _ = qbn.rope_frequencies(64)
    assert f[0] == plain[0] and math.isclose(f[-1], plain[-1] / scale, rel_tol=1e-12)
