"""Cross entropy over a vocabulary: the forward's sums over many channels leave the tensor core on the way.

The tensor core's additions cut off: a logit's running sum S loses, always towards 0, half a unit of its last place with each
of its C / 16 steps, 0.7 u |S| on average with u = 2^-24.  Logits of deviation s = 2.5; those that the log-sum-exp is made of lie
about s^2 = 6.25.  In one go |S| is 3.4 on the way to such a one: 256 steps of 0.7 u 3.4 are 3.6e-5, 3e-6 of a loss of 11.  In eight
sums of 512 channels |S| is 0.65 on the way, and 256 steps of 0.7 u 0.65 are 7e-6, 6e-7 of the loss; the given logit's own eight
sums differ in sign and add less, the last roundings 2 u = 1.2e-7.  Together the error's norm is below 8e-7 of the loss's.
"""
import pytest
import torch

import attention_kl_divergence_streamkl_gb300 as skl
from tests.test_gpu_vocab_xent import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("R,C,V", [(512, 4096, 8192), (40, 4096, 32000)])
def test_the_loss_of_many_channels(R, C, V, dtype):
    h, w, t = inputs(R, C, V, dtype, 41, none=0.0)
    loss, lse = skl.vocab_xent_fwd(h, w, t)
    z = torch.cat([h.double() @ x.double().T for x in w.split(8192)], 1)
    ref = torch.logsumexp(z, -1) - z.gather(1, t[:, None])[:, 0]
    assert 8 < float(ref.mean()) < 14 and 2 < float(z.std()) < 3
    assert float((loss.double() - ref).norm() / ref.norm()) <= 8e-7
