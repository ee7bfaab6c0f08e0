"""GPU tests of the gated delta rule's step at its limits."""
import pytest
import torch

import chunked_linear_scan_amd as cls

pytestmark = pytest.mark.gpu


def test_step_of_very_many_rows():
    """2^26 rows of states (2 GiB): each sequence as on its own."""
    nb, H, dk, dv = 1 << 14, 16, 8, 256
    g = torch.Generator(device="cuda").manual_seed(60)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    h = rn(nb, H, dv, dk)
    q, k = (torch.nn.functional.normalize(rn(nb, 1, dk), dim=-1).bfloat16() for _ in range(2))
    v, gl, beta = rn(nb, H, dv).bfloat16(), -rn(nb, H).abs(), torch.sigmoid(rn(nb, H))
    for part in (slice(0, 3), slice(nb // 2, nb // 2 + 1), slice(nb - 5, nb)):
        want_h = h[part].clone()
        want = cls.gated_delta_step(want_h, *(t[part] for t in (q, k, v, gl, beta)))
        before = h[part].clone()
        every = cls.gated_delta_step(h, q, k, v, gl, beta)
        assert torch.equal(every[part], want) and torch.equal(h[part], want_h) and not torch.equal(before, want_h)
