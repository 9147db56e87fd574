"""A workspace sized for N tokens serves every call with fewer: its size never falls as N grows
(a layer allocates for its largest batch and runs all others in the same memory).  Host only."""
import pytest

from mixture_experts_layer_50_b200 import _native as nat

SHAPES = [
    dict(d=2048, E=128, k=8, F=768),
    dict(d=7168, E=384, k=8, F=2048, n_shared=1),
    dict(d=1024, E=64, k=2, F=512),
    dict(d=4096, E=8, k=2, F=14336),
    dict(d=64, E=300, k=4, F=64),           # one slice of columns: the router is never cut
    dict(d=136, E=1024, k=1, F=64),
    dict(d=256, E=16, k=2, F=64, dtype=1),  # fp32
]


@pytest.mark.parametrize("shape", SHAPES)
def test_never_smaller_for_more_tokens(shape):
    last = 0
    for n in range(1, 2600):
        size = nat.moe_workspace_size(nat.make_config(n, **shape))
        assert size >= last, n
        last = size
    for n in (4096, 5000, 8192, 8193, 20000, 70000):
        size = nat.moe_workspace_size(nat.make_config(n, **shape))
        assert size >= last, n
        last = size


@pytest.mark.parametrize("shape", SHAPES[:3])
def test_never_smaller_for_more_capacity(shape):
    last = 0
    for c in range(0, 3000, 7):
        size = nat.moe_workspace_size(nat.make_config(200, capacity=c, **shape))
        assert size >= last, c
        last = size


@pytest.mark.parametrize("shape", SHAPES[:3])
@pytest.mark.parametrize("world", [1, 2, 3])
def test_a_rank_has_room_for_its_own_smaller_batches(shape, world):
    for most in (513, 1025, 1500):
        room = nat.moe_ep_workspace_size(nat.make_config(most, **shape), world)
        assert room >= max(nat.moe_workspace_size(nat.make_config(n, **shape)) for n in range(1, most + 1))


@pytest.mark.gpu
def test_a_smaller_batch_stays_in_its_workspace(cuda_dev):
    import torch

    d, E, k, F, most = 2048, 128, 8, 64, 1025
    room = nat.moe_workspace_size(nat.make_config(most, d, E, k, F))
    buf = torch.full((room + 256 + (8 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    start = -buf.data_ptr() % 256
    ws, behind = buf[start:start + room], buf[start + room:]
    nat.moe_workspace_init(ws)
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: (torch.randn(s, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    W_g, W_gu, W_down = r(E, d), r(E, 2 * F, d), r(E, d, F)
    for n in (1025, 1024, 897, 640):
        x, y = r(n, d), torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
        cfg = nat.make_config(n, d, E, k, F)
        logits = torch.empty(n, E, device="cuda")
        nat.moe_forward(cfg, x=x, W_g=W_g, W_gu=W_gu, W_down=W_down, y=y, route_out=dict(logits=logits), ws=ws)
        loss = torch.empty(1, device="cuda")
        ids = torch.argsort(logits, descending=True)[:, :k].to(torch.int32)
        nat.moe_balance_loss(cfg, logits=logits, ids=ids, alpha=1.0, loss=loss, ws=ws)
        assert nat.moe_check_status(ws) == 0
        assert bool((behind == 0x5A).all()), n
        want = torch.empty_like(y)
        nat.moe_forward(cfg, x=x, W_g=W_g, W_gu=W_gu, W_down=W_down, y=want, ws=nat.alloc_workspace(cfg))
        assert torch.equal(y, want), n
