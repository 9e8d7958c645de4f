"""A layer over microscaled 4-bit weights, as a serving step runs it with LoRA adapters in between: router, counts and
balance loss, both routings, the rows to 4 bits, gate_up, its delta, the activation to 4 bits, down, its delta, combine. Each
step is compared with its definition in 64 bits on what the step before left.

Tolerances. Products: as in test_moe_mx4_gpu.py. A delta: x A of K terms and s B of r in fp32 in any order, the scale and
the addition, (K + r + 3) 2^-24 of the sums' magnitudes, and half a bf16 step of the row. The combine: topk + 1 fp32
roundings and half a step."""
import numpy as np
import pytest
import torch

from tests import mx4_defs as d
from virtual_expert_routed_amd import binding as mb

pytestmark = pytest.mark.gpu

U, HALF = 2.0 ** -24, 2.0 ** -8


def value(q, s):
    return torch.from_numpy(d.decode(q.cpu().numpy(), s.cpu().numpy())).cuda()


def near(got, ref, slack):
    return bool(((got.double() - ref).abs() <= slack * (1 + HALF) + HALF * ref.abs()).all())


class Layer:
    def __init__(self, M, E, topk, S, H, I, r, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def n(*shape, sigma=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * sigma).bfloat16()

        self.M, self.E, self.topk, self.S, self.H, self.I, self.r = M, E, topk, S, H, I, r
        self.numel, self.V, self.block = M * topk, E * S, 64
        self.logits, self.x = n(M, E, sigma=2.0), n(M, H)
        self.mask = torch.rand(M, generator=g, device="cuda") < 0.9
        self.lora = torch.randint(-1, S, (M,), generator=g, device="cuda", dtype=torch.int32)
        self.scale = torch.rand(S, generator=g, device="cuda") + 0.5
        self.W1 = mb.mol_mx4_quantize(n(E, 2 * I, H, sigma=0.06))
        self.W2 = mb.mol_mx4_quantize(n(E, H, I, sigma=0.06))
        self.A1, self.B1 = n(self.V, 2 * r, H, sigma=0.05), n(self.V, 2 * I, r, sigma=0.05)
        self.A2, self.B2 = n(self.V, r, I, sigma=0.05), n(self.V, H, r, sigma=0.05)
        self.gate_up = torch.zeros(self.numel, 2 * I, dtype=torch.bfloat16, device="cuda")
        self.down = torch.zeros(self.numel, H, dtype=torch.bfloat16, device="cuda")
        self.bws = mb.new_router_balance_workspace(M, E, "cuda")
        self.dws = mb.new_delta_workspace(self.numel, 2 * r, self.V, self.block, "cuda")

    def step(self, look=lambda name, *tensors: None):
        t = self
        ids, w = mb.mol_router_topk(t.logits, t.topk)
        loss, counts, _ = mb.mol_router_balance(t.logits, ids, alpha=0.01, token_mask=t.mask, workspace=t.bws)
        look("counts", ids, counts, loss)
        base = mb.mol_align_block_size(ids, None, t.E, 1, t.block)
        virt = mb.mol_align_block_size(ids, t.lora, t.E, t.S, t.block)
        q, s = mb.mol_mx4_quantize(t.x)
        mb.mol_moe_gemm_mx4(q, t.topk, *t.W1, *base, t.numel, t.block, t.gate_up, x_scales=s)
        look("gate_up", ids, q, s, t.gate_up)
        mb.mol_lora_delta(t.x, t.topk, t.A1, 2, t.B1, t.scale, t.E, *virt, t.numel, t.V, t.block, t.gate_up, t.dws)
        look("gate_up delta", ids, t.gate_up)
        q, s = mb.mol_mx4_quantize(t.gate_up, mb.MOL_ACT_SILU_MUL)
        look("act", t.gate_up, q, s)
        mb.mol_moe_gemm_mx4(q, 1, *t.W2, *base, t.numel, t.block, t.down, x_scales=s)
        look("down", ids, q, s, t.down)
        h = mb.mol_mx4_dequantize(q, s)
        mb.mol_lora_delta(h, 1, t.A2, 1, t.B2, t.scale, t.E, *virt, t.numel, t.V, t.block, t.down, t.dws)
        look("down delta", ids, h, t.down)
        y = mb.mol_moe_combine(t.down, ids, w, t.E)
        look("combine", ids, w, t.down, y)
        return loss, counts, y


@pytest.mark.parametrize("M,E,topk,S,H,I,r,seed", [(1, 8, 2, 2, 256, 128, 16, 1), (23, 16, 4, 3, 512, 96, 32, 2),
                                                   (300, 4, 2, 2, 384, 160, 8, 3), (2100, 16, 4, 1, 256, 1664, 16, 4)])
def test_each_step(M, E, topk, S, H, I, r, seed):
    t = Layer(M, E, topk, S, H, I, r, seed)
    rows = torch.arange(t.numel, device="cuda")
    before = {}

    def product(name, ids, x, W, s, out):
        flat = ids.reshape(-1)
        for e in range(E):
            p = rows[flat == e]
            w = value(W[e], s[e])
            assert near(out[p], x[p] @ w.t(), (x.shape[1] + 1) * U * (x[p].abs() @ w.abs().t())), name
        before[name] = out.clone()

    def delta(name, ids, x, A, B, slices, out):
        slot = t.lora.repeat_interleave(topk).long()
        flat = ids.reshape(-1).long()
        n = out.shape[1] // slices
        for v in range(t.V):
            p = rows[(slot == v // E) & (flat == v % E)]
            if not p.numel():
                continue
            a, b, c = A[v].double(), B[v].double(), float(t.scale[v // E])
            s, sm = x[p] @ a.t(), x[p].abs() @ a.abs().t()
            d_ = torch.cat([s[:, i * r:(i + 1) * r] @ b[i * n:(i + 1) * n].t() for i in range(slices)], 1) * c
            dm = torch.cat([sm[:, i * r:(i + 1) * r] @ b[i * n:(i + 1) * n].abs().t() for i in range(slices)], 1) * c
            ref = before[name][p].double() + d_
            # (prefill batches take bf16 matrix-core tiles, which multiply s as bf16 terms: their own tests' bound)
            wide = 1e-2 * float(d_.abs().max()) if t.numel >= 4096 else 0.0
            assert near(out[p], ref, (x.shape[1] + r + 3) * U * (dm + before[name][p].double().abs()) + wide), name
        assert torch.equal(out[slot < 0], before[name][slot < 0])

    def look(name, *a):
        if name == "counts":
            ids, counts, loss = a
            live = ids[t.mask].reshape(-1).long()
            assert torch.equal(counts[:E].long(), torch.bincount(live, minlength=E)) and int(counts[E]) == int(t.mask.sum())
            p = torch.softmax(t.logits[t.mask].double(), dim=1).sum(0)
            n = max(int(counts[E]), 1)
            assert abs(float(loss) - 0.01 * E / (topk * n * n) * float((counts[:E].double() * p).sum())) <= 2.0 ** -16 * float(loss) + 1e-30
        elif name == "gate_up":
            ids, q, s, out = a
            rq, rs = d.encode(t.x.double().cpu().numpy())
            assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
            product(name, ids, value(q, s).repeat_interleave(topk, dim=0), *t.W1, out)
        elif name == "gate_up delta":
            delta("gate_up", a[0], t.x.double().repeat_interleave(topk, dim=0), t.A1, t.B1, 2, a[1])
        elif name == "act":
            rq, rs = d.encode(d.silu_mul(a[0].double().cpu().numpy()))
            assert np.array_equal(a[1].cpu().numpy(), rq) and np.array_equal(a[2].cpu().numpy(), rs)
        elif name == "down":
            ids, q, s, out = a
            product(name, ids, value(q, s), *t.W2, out)
        elif name == "down delta":
            delta("down", a[0], a[1].double(), t.A2, t.B2, 1, a[2])
        else:
            ids, w, rows_, y = a
            z = rows_.double().view(M, topk, H) * w.double().unsqueeze(2)
            assert near(y, z.sum(1), (topk + 1) * U * z.abs().sum(1))

    t.step(look)


@pytest.mark.parametrize("M", [23, 1200])
def test_the_step_in_a_graph(M):
    t = Layer(M, 16, 4, 2, 256, 96, 16, 7)
    want = t.step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = t.step()
    for turn in range(3):
        t.x.mul_(0.75 + turn), t.logits.copy_(t.logits.roll(1, dims=1)), t.lora.copy_(t.lora.roll(1))
        t.gate_up.zero_(), t.down.zero_()
        want = [v.clone() for v in t.step()]
        t.gate_up.zero_(), t.down.zero_()
        for v in out:
            v.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
