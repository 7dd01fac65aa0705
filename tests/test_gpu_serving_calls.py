"""Calls of the paged decode, the page operations and the norms that their documentation allows or
refuses at its edges: views, refusals that leave everything as it was, optional outputs, every
dispatch. Error bounds are counted as in serving_ref.py."""
import pytest
import torch

import gated_deltanet_mixer_causal_b200 as gdn
from test_gpu_paged import case, ints

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def test_expanded_tensors_are_refused(cuda_device):
    """One token, gate, gradient buffer or page in place of many has the memory of one."""
    dev = cuda_device
    c = case(dev, 4, 1, 1, 2, 16, FP, FP, 6, seed=1)
    args = dict(x=c["x"], conv_w=c["conv_w"], conv_pool=c["conv"], state_pool=c["state"], read_pages=ints([0, 1, 2, 3], dev),
                g=c["g"], beta=c["beta"], Hk=1)
    gate = dict(z=torch.zeros(1, 1, 2, 16, device=dev).expand(4, 1, 2, 16), norm_w=torch.ones(16, device=dev))
    kept = c["state"].clone(), c["conv"].clone()
    for kw in (dict(x=c["x"][:1].expand(4, 1, 64)), gate, dict(conv_pool=c["conv"][:1].expand(6, 3, 64)),
               dict(state_pool=c["state"][:1].expand(6, 2, 16, 16))):
        with pytest.raises(ValueError, match="share memory"):
            gdn.gdn_decode_paged(**{**args, **kw})
    assert torch.equal(kept[0], c["state"]) and torch.equal(kept[1], c["conv"])
    o = torch.zeros(5, 2, 16, device=dev)
    one = torch.zeros(1, 2, 16, device=dev).expand(5, 2, 16)
    w = torch.ones(16, device=dev)
    for call in (lambda: gdn.gdn_gated_norm(o, one, w), lambda: gdn.gdn_gated_norm_bwd(o, one, w, o),
                 lambda: gdn.gdn_gated_norm_bwd(o, o, w, o, dz=one)):
        with pytest.raises(ValueError, match="share memory"):
            call()
    template, pool = torch.ones(1, 16, device=dev), torch.zeros(6, 16, device=dev)
    lists, refs = ints([0, 5], dev), ints([1, 0, 0, 0, 0, 0], dev)
    for call in (lambda: gdn.gdn_pages_copy(template.expand(6, 16), lists, lists, dst_pool=pool),
                 lambda: gdn.gdn_pages_copy(pool, lists, lists, dst_pool=template.expand(6, 16)),
                 lambda: gdn.gdn_pages_fork(refs, ints([0], dev), template.expand(6, 16)),
                 lambda: gdn.gdn_pages_compact(refs, None, template.expand(6, 16))):
        with pytest.raises(ValueError, match="share memory"):
            call()
    assert (pool == 0).all() and refs.tolist() == [1, 0, 0, 0, 0, 0]
