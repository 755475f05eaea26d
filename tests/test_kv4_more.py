"""More of the decode over a 4-bit cache."""
import numpy as np
import pytest

import oracle
from test_kv4 import Case, f64, fd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sms", [0, 1])
@pytest.mark.parametrize("G,d", [(1, 64), (2, 128), (4, 128), (8, 64), (16, 128)])
def test_sequences_without_any_weight(fd, G, d, sms):  # noqa: F811
    """Every score of a sequence overflows to -inf: out is 0 and lse -inf, as for one without tokens,
    whether a CTA has the pair alone or shares it, and on the one-CTA-per-partial kernel too."""
    import torch
    c = Case(fd, "bf16_e2m1kv", d, G, 2, [3000, 100, 16, 40], [3, 1, 1, 1], seed=33, garbage=False)
    c.q = torch.full_like(c.q, 1e38)
    k = np.zeros(tuple(c.k.shape), np.uint8)
    k[:, :, :8 * d], k[:, :, 8 * d:] = 0xFF, 0x7E            # -2688 everywhere
    k[-1] = 0                                                # but in the last block of the last sequence
    c.k = torch.from_numpy(k).cuda()
    c.ref[0][:3], c.ref[1][:3] = 0, -np.inf
    c.ref[0][3] = np.repeat(c.values[1][-8:].mean(0), G, axis=0)
    c.ref[1][3] = np.log(8)
    for flags in (0, fd.FD_PLAN_TWO_LAUNCH, fd.FD_PLAN_NO_CLUSTER):
        c.check(*c.run(c.decoder(flags=flags, num_sms=sms)))
