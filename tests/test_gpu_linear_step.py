"""llsa_linear_step on the GPU against the fp64 reference, its pool rules, and the operators of a
decode loop together.

Tolerance: fp32 throughout (the product l S + k v and D products and sums for o), so with the
terms' magnitudes A the error is below (D + 8) 2^-24 A < 2^-16 A; a bf16 output adds 2^-8 of its
value."""
import numpy as np
import pytest
import torch

import log_linear_hierarchical_b200 as llsa
from oracle import sequence_ops as so

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def num(t):
    return t.detach().double().cpu().numpy()


def make(B, H, D, P, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + B + H + D)
    q, k, v = (torch.randn(B, H, D, device="cuda", generator=g).to(dtype) for _ in range(3))
    pool = torch.randn(P, H, D, D, device="cuda", generator=g)
    a = torch.tensor([[-0.02, 0.0, -0.7, -30.0][h % 4] for h in range(H)], device="cuda")
    return q, k, v, pool, a


def check(o, pool, q, k, v, old, a, slots, out_slots):
    D = q.shape[-1]
    args = [num(t) for t in (q, k, v)]
    wo, wp = so.linear_step(*args, num(a), D ** -0.5, num(old), slots, out_slots)
    ao, ap = so.linear_step(*(np.abs(t) for t in args), num(a), D ** -0.5, np.abs(num(old)), slots, out_slots)
    assert (np.abs(num(pool) - wp) <= 2.0 ** -16 * ap).all()
    assert (np.abs(num(o) - wo) <= 2.0 ** -16 * ao + (2.0 ** -8 * np.abs(wo) if o.dtype == BF else 0)).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,H,D", [(1, 1, 64), (3, 5, 64), (2, 4, 128), (33, 2, 128)])
def test_in_place_and_slots(dtype, B, H, D):
    q, k, v, pool, a = make(B, H, D, 2 * B + 1, dtype)
    old = pool.clone()
    o = llsa.llsa_linear_step(q, k, v, a, pool)
    check(o, pool, q, k, v, old, a, range(B), range(B))
    old = pool.clone()
    slots = torch.randperm(2 * B + 1, device="cuda").to(torch.int32)
    if B > 1:
        slots[1] = -1
    o = llsa.llsa_linear_step(q, k, v, a, pool, slots=slots[:B].contiguous(), out_slots=slots[B:2 * B].contiguous())
    check(o, pool, q, k, v, old, a, slots[:B].tolist(), slots[B:2 * B].tolist())
    old, out = pool.clone(), torch.full_like(q, 7.0)
    assert llsa.llsa_linear_step(q, k, v, a, pool, slots=slots[:B].contiguous(), out=out) is out
    check(out, pool, q, k, v, old, a, slots[:B].tolist(), slots[:B].tolist())
    assert llsa.llsa_device_status() == 0


def test_colliding_and_outside_slots_take_no_part_and_are_recorded():
    q, k, v, pool, a = make(6, 2, 64, 8, F32)
    i32 = lambda *x: torch.tensor(x, device="cuda", dtype=torch.int32)  # noqa: E731
    # row 2 repeats row 0's slot; row 4 is outside the pool; row 5 writes what row 1 reads
    old = pool.clone()
    o = llsa.llsa_linear_step(q, k, v, a, pool, slots=i32(3, 1, 3, 0, 8, 5), out_slots=i32(3, 2, 3, 0, 8, 1))
    assert llsa.llsa_device_status() == 5
    check(o, pool, q, k, v, old, a, [3, 1, -1, 0, -1, -1], [3, 2, -1, 0, -1, -1])
    # an inactive row blocks nobody; a row may not read what an earlier row writes
    old = pool.clone()
    o = llsa.llsa_linear_step(q, k, v, a, pool, slots=i32(-1, 3, 4, 7, 6, 5), out_slots=i32(3, 3, 2, 4, 0, 6))
    assert llsa.llsa_device_status() == 5
    check(o, pool, q, k, v, old, a, [-1, 3, 4, -1, 6, -1], [-1, 3, 2, -1, 0, -1])
    assert llsa.llsa_device_status() == 0


def test_views_and_streams():
    q, k, v, pool, a = make(4, 3, 64, 4, BF)
    wide = torch.stack((q, k, v), 2)                    # [B, H, 3, D]: strided rows are copied
    p2, p3 = pool.clone(), pool.clone()
    o = llsa.llsa_linear_step(q, k, v, a, pool)
    assert torch.equal(llsa.llsa_linear_step(wide[:, :, 0], wide[:, :, 1], wide[:, :, 2], a, p2), o)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o3 = llsa.llsa_linear_step(wide[:, :, 0], wide[:, :, 1], wide[:, :, 2], a, p3, stream=s)
    s.synchronize()
    assert torch.equal(o3, o) and torch.equal(p2, pool) and torch.equal(p3, pool)


def test_refusals():
    q, k, v, pool, a = make(2, 2, 64, 2, F32)
    for call in (lambda: llsa.llsa_linear_step(q, k, v, a, pool.transpose(2, 3)),
                 lambda: llsa.llsa_linear_step(q, k, v, a, pool.cpu()),
                 lambda: llsa.llsa_linear_step(q, k, v, a, pool, slots=torch.zeros(2, device="cuda", dtype=torch.int64)),
                 lambda: llsa.llsa_linear_step(q, k, v, a, pool, slots=torch.zeros(3, device="cuda", dtype=torch.int32)),
                 lambda: llsa.llsa_linear_step(q.requires_grad_(), k, v, a, pool)):
        with pytest.raises(ValueError):
            call()
    q = q.detach()
    with pytest.raises(llsa.LLSAError):
        llsa.llsa_linear_step(q, k, v, a, pool[:1])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_prompt_then_tokens_is_the_whole_sequence(dtype):
    """Rotated prompts of unequal lengths, then rotated tokens one at a time over the pool, against
    the reference on each whole rotated sequence."""
    B, H, D, N, T = 3, 2, 64, 200, 5
    lengths = [200, 1, 77]
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(B, N + T, H, D, device="cuda", generator=g).to(dtype) for _ in range(3))
    f, scale = llsa.llsa_rotary_frequencies(32, scaling="yarn", factor=2.0, original_length=64, device="cuda")
    a = torch.tensor([-0.05, -0.003], device="cuda")
    tr = lambda x: x[:, :N].transpose(1, 2)  # noqa: E731
    q1, k1 = llsa.llsa_rotary(tr(q), tr(k), None, f, first=16, scale=scale)
    L = torch.tensor(lengths, device="cuda", dtype=torch.int32)
    o, pool = llsa.llsa_linear_attention(q1, k1, tr(v), a, lengths=L, return_state=True)
    rows, toks = [], []
    for t in range(T):
        at = (L.long() + t)[:, None]
        pick = lambda x: x[torch.arange(B, device="cuda"), at[:, 0]].unsqueeze(2)  # noqa: E731  [B, H, 1, D]
        qt, kt = llsa.llsa_rotary(pick(q), pick(k), at, f, first=16, scale=scale)
        toks.append((qt, kt, pick(v)))
        rows.append(llsa.llsa_linear_step(qt[:, :, 0], kt[:, :, 0], pick(v)[:, :, 0], a, pool))
    for b, n in enumerate(lengths):
        x = [np.concatenate([num(p)[b:b + 1, :, :n]] + [num(t[i])[b:b + 1] for t in toks], axis=2)
             for i, p in enumerate((q1, k1, tr(v)))]
        want, S, _ = so.linear_forward(*x, num(a), D ** -0.5)
        size, AS, _ = so.linear_forward(*(np.abs(t) for t in x), num(a), D ** -0.5)
        got = np.concatenate([num(o)[b:b + 1, :, :n]] + [num(r)[b:b + 1, :, None] for r in rows], axis=2)
        # as the prompt's tolerance: operands and results rounded to bf16 (2^-8 each) or fp32 sums
        tol = 1.02 * (2.0 ** -8 * (size + np.abs(want)) + 2.0 ** -16 * size) if dtype == BF else 2.0 ** -17 * size
        assert (np.abs(got - want) <= tol).all()
        assert (np.abs(num(pool)[b:b + 1] - S) <= (2.0 ** -16 + 2.0 ** -17) * AS).all()


def test_a_hybrid_block_trains_and_replays():
    """Rotary into the sparse attention and into linear attention side by side: gradients of the sum
    equal the sum of the layers' own, eagerly and from a captured graph."""
    B, H, N, D = 1, 2, 1024, 64
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k, v, do = (torch.randn(B, H, N, D, device="cuda", generator=g).to(BF) for _ in range(4))
    f, _ = llsa.llsa_rotary_frequencies(64, device="cuda")
    a = torch.tensor([-0.01, -0.1], device="cuda")
    leaves = [t.requires_grad_() for t in (q, k, v)]

    def block(sparse=True, linear=True):
        q1, k1 = llsa.llsa_rotary(q, k, None, f)
        out = []
        if sparse:
            out.append(llsa.llsa_attention(q1, k1, v, topk=8, levels=1))
        if linear:
            out.append(llsa.llsa_linear_attention(q1, k1, v, a))
        return [o.detach() for o in out], torch.autograd.grad(out, leaves, [do] * len(out))

    (os_, ol), both = block()
    (o1,), g1 = block(linear=False)
    (o2,), g2 = block(sparse=False)
    assert torch.equal(os_, o1) and torch.equal(ol, o2)
    for x, y, z in zip(both, g1, g2):
        # the sum is made in bf16 before the inverse rotation or after it: three roundings of values
        # of at most |y| + |z| and their rotated pair's
        bound = (y.abs().float() + z.abs().float()).amax(-1, keepdim=True)
        assert ((x.float() - y.float() - z.float()).abs() <= 4 * 2.0 ** -8 * bound).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (h1, h2), hg = block()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h1, os_) and torch.equal(h2, ol) and all(torch.equal(x, y) for x, y in zip(hg, both))
    assert llsa.llsa_device_status() == 0
