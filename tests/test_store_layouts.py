"""Layouts of the slot-mapped store's tokens: strides count only where there is more than one element to step over."""

import pytest
import torch


@pytest.fixture(scope="module")
def kv():
    from calibration_free_kv_gb300 import build
    build.build()
    from calibration_free_kv_gb300 import kvarn
    return kvarn


def _layouts(device="cpu"):
    """(k, v) whose strides differ in dimensions of size 1 only."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 12, 64, generator=g).half().to(device)
    fresh = lambda t: torch.empty(t.shape, dtype=t.dtype, device=device).copy_(t)  # noqa: E731
    one = x[1:2, 4:6], fresh(x[2:3, 7:9])                                        # one token, of two tensors
    odd = x[1:2, 4:6], x.flatten()[8:].as_strided((1, 2, 64), (3, 64, 1))        # its token stride means nothing
    head = x[:, 3:4], x.flatten()[16:].as_strided((3, 1, 64), (12 * 64, 5, 1))   # one head
    both = x[:1, :1], fresh(x[2:, 3:4])
    return {"one token": one, "odd stride": odd, "one head": head, "one of each": both}


@pytest.mark.parametrize("name", list(_layouts()))
def test_taken_on_the_host(kv, name):
    k, v = _layouts()[name]
    slots, pool = torch.zeros(k.shape[0], dtype=torch.int64), torch.zeros(1, k.shape[1], 2, 128, 64, dtype=torch.float16)
    assert k.stride() != v.stride()
    with pytest.raises(ValueError, match="CUDA"):  # refused for being on the host, not for the layout
        kv.fp16_store(k, v, slots, pool)


def test_other_strides_are_refused(kv):
    x = torch.zeros(3, 12, 64, dtype=torch.float16)
    slots, pool = torch.zeros(3, dtype=torch.int64), torch.zeros(1, 2, 2, 128, 64, dtype=torch.float16)
    for k, v in ((x[:, :2], x[:, :2].contiguous()), (x[:, :2], x[:, :4:2]), (x[:1, :2], x[:1, :4:2]),
                 (x[:, :1], x[:, :1].contiguous()), (x[..., ::2][:, :2], x[..., ::2][:, :2])):
        with pytest.raises(ValueError, match="matching strides"):
            kv.fp16_store(k, v, slots[:k.shape[0]], pool)


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(_layouts()))
def test_stored(kv, name):
    k, v = _layouts("cuda")[name]
    tokens, heads, dim = k.shape
    slots = torch.arange(tokens, device="cuda") * 100 + 27
    pool = torch.zeros(3, heads, 2, 128, dim, dtype=torch.float16, device="cuda")
    kv.fp16_store(k, v, slots, pool)
    want = torch.zeros_like(pool)
    for t, s in enumerate(slots.tolist()):
        want[s // 128, :, 0, s % 128], want[s // 128, :, 1, s % 128] = k[t], v[t]
    assert torch.equal(pool, want)


@pytest.mark.gpu
def test_device_of_a_tensor_is_told(kv):
    # as a call on the second GPU would find it
    t = torch.zeros(2, 3, device="cuda")
    with pytest.raises(ValueError, match="scores is on cuda:0, the call's first tensor on cuda:1"):
        kv._arg("scores", t, 1, torch.float32, (2, 3))
