"""Every step and centre that a 16-bit extreme can give, and codes whose quotients are near a
half, equal to the definition to the bit."""
import pytest
import torch

import kv_reference as ref
from test_gpu_kv_cache import BF, FP, same_bits

pytestmark = pytest.mark.gpu


def write_and_compare(x, G):
    """x [tokens, 1, 64]: steps, centres and stored values of keys and values."""
    from moe_expert_layer_sorted_gb300 import KVCache
    n, dtype = x.shape[0], x.dtype
    c = KVCache.allocate(-(-n // 256), kv_heads=1, head_dim=64, page_size=256, group_size=G, dtype=dtype)
    at = dict(table=torch.arange(-(-n // 256), dtype=torch.int32, device="cuda")[None],
              lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
    v = x.flip(0).contiguous()
    c.append(x[None], v[None], **at)
    ko, vo = torch.empty_like(x)[None], torch.empty_like(x)[None]
    c.read(ko, vo, **at)
    params = c.pages[0, :, 0].flatten(0, 1)[:, 16 * 64:].contiguous().view(dtype).view(-1, 2, 16, 64 // G, 2)
    for m, (y, out) in enumerate(((x, ko), (v, vo))):
        _, s, cc = ref.quantise(y, G)
        par = params[:, m].flatten(0, 1)[:n]
        assert same_bits(par[..., 0], s[:, 0]) and same_bits(par[..., 1], cc[:, 0])
        assert same_bits(out[0], ref.values(y, G).float().to(dtype))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("low", ["zero", "opposite", "half"])
def test_steps_of_every_value(dtype, low):
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(dtype)
    x = x[torch.isfinite(x)][:63488].cuda()
    other = {"zero": torch.zeros_like(x), "opposite": -x, "half": (x.float() / 2).to(dtype)}[low]
    g = torch.where(torch.arange(32, device="cuda") % 3 == 0, x[:, None], other[:, None])
    write_and_compare(g.view(-1, 1, 64).contiguous(), 32)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("kind", ["whole", "scaled", "wide"])
def test_quotients_near_a_half(dtype, kind):
    """Whole numbers whose step is a whole number too (ties in every row), the same times powers
    of two down to the subnormals, and any values."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n = 1 << 16
    if kind == "wide":
        x = torch.randn(n, 1, 64, generator=g, device="cuda") * torch.exp2(torch.randint(-20, 15, (n, 1, 1), generator=g, device="cuda").float())
    else:
        step = torch.randint(1, 9, (n, 1, 1), generator=g, device="cuda")
        x = torch.randint(0, 1 << 20, (n, 1, 64), generator=g, device="cuda") % (15 * step + 1) - 7 * step
        x[:, 0, ::32], x[:, 0, 1::32] = (-7 * step)[:, 0], (8 * step)[:, 0]  # step / 1: quotients at halves where it is even
        x = x.float()
        if kind == "scaled":
            x = x * torch.exp2(torch.randint(-22 if dtype == FP else -130, 4, (n, 1, 1), generator=g, device="cuda").float())
    write_and_compare(x.to(dtype), 32)
    write_and_compare(x.to(dtype), 64)
