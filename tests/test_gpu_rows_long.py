"""GPU: the expert MLP and the adapter linear where a tile's activations pass
through LDS in slices: many groups of input channels for every tile height,
with slices that do not divide them, several columns to a wavefront, rows that
leave parts of a tile empty, and columns past the last strip.

Tolerances as in test_gpu_rows.py, whose definitions and checks these use.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_rows import (acts, check_lora, check_moe, lora_case, moe_case, moe_ref, pack,  # noqa: E402
                           w4)  # noqa: F401

MOE = [
    # M, k, E, I, K: up to 16, 32 and 64 rows a tile
    (20, 2, 8, 128, 4352), (12, 1, 3, 4224, 256), (23, 2, 6, 4352, 4224),
    (60, 2, 8, 128, 2304), (60, 2, 8, 2304, 128), (41, 3, 7, 2176, 2432),
    (100, 3, 6, 128, 1280), (100, 3, 6, 1152, 128), (75, 4, 8, 1408, 1664), (130, 2, 5, 1280, 2688),
]


@pytest.mark.parametrize("M,k,E,I,K", MOE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_moe_sliced(w4, M, k, E, I, K, dtype):  # noqa: F811
    x, up, down, ids, wt = moe_case(M + K, M, k, E, I, K, dtype, drop=0.2, skew=M % 2 == 1)
    y = w4.moe_mlp(x, *pack(w4, up, down, E), ids, wt)
    check_moe(y, *moe_ref(x, up, down, ids, wt, E))


@pytest.mark.parametrize("P", [4095, 4096, 4097, 9000])
@pytest.mark.parametrize("E,k", [(5, 1), (200, 3)])
def test_moe_many_pairs(w4, P, E, k):  # noqa: F811
    """Pairs counted by one workgroup and by several, with experts of no pair
    and one of very many, slots of other experts, repeated ids in a token."""
    M, I, K = P // k, 128, 128
    x, up, down, ids, wt = moe_case(P, M, k, E, I, K, torch.bfloat16, drop=0.1, skew=True)
    g = torch.Generator(device="cuda").manual_seed(P)
    ids = torch.where(torch.rand(M, k, generator=g, device="cuda") < 0.3, 2, ids).contiguous()
    y = w4.moe_mlp(x, *pack(w4, up, down, E), ids, wt)
    check_moe(y, *moe_ref(x, up, down, ids, wt, E))


LORA = [
    # M, K, N, L, R, seg: two, three and four 16-row fragments, K in two slices
    (20, 4608, 32784, 3, 8, 1), (45, 2816, 32784, 4, 72, 3), (61, 2304, 32784, 5, 32, 1),
    # rows taken in the order of their adapters: more adapters than buckets of that order, few
    # rows over many channels, ranks past 64, all with K whole and in slices
    (90, 256, 272, 2000, 8, 1), (300, 1152, 272, 1500, 16, 1), (64, 256, 18960, 64, 64, 1),
    (700, 256, 4112, 9, 72, 1), (300, 1024, 1040, 16, 128, 1), (517, 384, 2064, 3, 128, 11),
    # 256 x 256 tiles past a whole round of the compute units: half tiles, an odd number of them
    (1000, 256, 17424, 6, 40, 1), (2048, 128, 9232, 4, 16, 300), (300, 384, 33040, 3, 8, 2),
    # eight wavefronts to a column, with rows that end inside the fragment
    (16, 3584, 2064, 5, 72, 1), (11, 1152, 3584, 16, 128, 1), (2, 4096, 4096, 2, 8, 1), (9, 4224, 2304, 4, 24, 1),
    # the single token: K whole, K split over workgroups, a long token, many channels
    (1, 3584, 3584, 3, 128, 1), (1, 18944, 3584, 2, 72, 1), (1, 8192, 512, 2, 8, 1), (1, 256, 50000, 2, 40, 1),
    (1, 36864, 256, 2, 16, 1),
]


@pytest.mark.parametrize("M,K,N,L,R,seg", LORA)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_lora_sliced(w4, M, K, N, L, R, seg, dtype):  # noqa: F811
    x, w, A, B, sc, ids = lora_case(M + N, M, K, N, L, R, dtype, seg)
    if M == 1:
        ids.clamp_(min=0)
    W = w4.pack_weights(*w)
    check_lora(w4.lora_linear(x, W, w4.LoraAdapters(A, B, sc), ids), x, w, A, B, sc, ids)
    if M == 1:
        ids.fill_(-1)
        check_lora(w4.lora_linear(x, W, w4.LoraAdapters(A, B, sc), ids), x, w, A, B, sc, ids)


def near_scores(g, M, E, kind):
    """Logits whose sigmoids, with the bias, lie next to each other: equal ones,
    neighbours in float32, and ones that round to one float32."""
    base = torch.randn(M, 1, generator=g, device="cuda")
    if kind == "equal":
        l = base.expand(M, E).clone()
    elif kind == "neighbours":
        l = base.repeat(1, E)
        step = torch.randint(0, 3, (M, E), generator=g, device="cuda").float()
        l = l * (1 + step * 2.0 ** -23)
    else:
        l = base + torch.rand(M, E, generator=g, device="cuda") * 1e-5
    return l.contiguous()


@pytest.mark.parametrize("kind", ["equal", "neighbours", "close"])
@pytest.mark.parametrize("E,n_groups,group_top", [(64, 1, 1), (96, 4, 2), (63, 7, 2), (250, 10, 2), (1023, 33, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_next_to_a_border(w4, kind, E, n_groups, group_top, score):  # noqa: F811
    """Choices that float32 scores cannot decide; the definition of
    test_gpu_rows.py decides them in 64 bits.  Sums of two scores that differ
    by less than 64-bit rounding cannot occur: the inputs are float32."""
    from test_gpu_rows import route_ref
    M, k = 9, 5
    g = torch.Generator(device="cuda").manual_seed(E)
    l = near_scores(g, M, E, kind)
    # a bias of a few values, exact in every sum
    bias = torch.randint(0, 2, (E,), generator=g, device="cuda").float() * 0.25
    if kind != "equal" and score == "softmax":
        # the 64-bit softmax of the definition and the kernel's may round the
        # last bit apart; spread the logits so that no choice hangs on it
        l = l + torch.arange(E, device="cuda") % 7 * 2.0 ** -12
    kw = dict(score=score, n_groups=n_groups, topk_groups=max(1, n_groups // 2), group_top=group_top,
              renormalize=True, scale=1.0)
    ids, w = w4.moe_route(l, k, bias=bias, **kw)
    rid, rw = route_ref(l, k, score, bias, n_groups, kw["topk_groups"], group_top, True, 1.0)
    if kind == "equal":
        assert torch.equal(ids.cpu(), rid)
    else:
        # the chosen values in order, as the definition's; equal values may sit
        # at other indices only where 64-bit scores agree to the last bits
        p = torch.softmax(l.double().cpu(), 1) if score == "softmax" else torch.sigmoid(l.double().cpu())
        c = p + bias.double().cpu()
        a, b = c.gather(1, ids.cpu().long()), c.gather(1, rid.long())
        assert ((a - b).abs() <= 2.0 ** -50).all()
    assert ((w.cpu().double() - rw).abs() <= (E + 16) * 2.0 ** -24 * rw.abs()).all()


def test_host_tensors_are_refused(w4):  # noqa: F811
    """A tensor in host memory, the workspace among them, never reaches a kernel."""
    x, w, A, B, sc, ids = lora_case(1, 4, 256, 272, 2, 8, torch.bfloat16)
    W, ad = w4.pack_weights(*w), w4.LoraAdapters(A, B, sc)
    host = torch.empty(w4.lora_linear_workspace_bytes(4, 272, 256, 2, 8), dtype=torch.uint8)
    for kw in (dict(workspace=host), dict(out=torch.empty(4, 272, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            w4.lora_linear(x, W, ad, ids, **kw)
    with pytest.raises(ValueError):
        w4.lora_linear(x, W, ad, ids.cpu())
    with pytest.raises(ValueError):
        w4.lora_linear(x.repeat(1, 2)[:, ::2], W, ad, ids)       # not contiguous
    xm, up, down, eid, wt = moe_case(1, 4, 2, 3, 128, 256, torch.bfloat16)
    ups = pack(w4, up, down, 3)
    with pytest.raises(ValueError):
        w4.moe_mlp(xm, *ups, eid, wt, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        w4.moe_mlp(xm, *ups, eid, wt.cpu())
    with pytest.raises(ValueError):
        w4.moe_route(torch.zeros(2, 8, device="cuda"), 2, bias=torch.zeros(8))
