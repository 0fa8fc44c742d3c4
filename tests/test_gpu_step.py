"""The operators between the token ids and the experts in a run, as a training
step uses them: embedding, dropout, layer norm, router, sort, dispatch, combine
and the layer norm after it, and back to the gradient of the table.

In fp32, against autograd in 64 bits with the same dropped elements and the
routing that the router chose.  Every stage adds at most some 2 * 128 * 2^-24 of
its values' size (sums along a row are counted as 128 additions deep, those over
the tokens of a table's row or a column as no deeper here), a dozen of them
forward and as many back: 24 * 2 * 128 * 2^-24 = 4e-4 of the size of what comes
out, the norms' and softmax's own derivatives being near 1 for these inputs."""
import pytest
import torch

import cast_transpose_gb300 as ct
import step_reference as ref

pytestmark = pytest.mark.gpu

F32, I32 = torch.float32, torch.int32
SEED, P, EPS, BALANCE, Z = 99, 0.2, 1e-5, 0.05, 0.01
MOST = 4e-4


class Step:
    """Buffers and parameters of a model's first block; run() is one step."""

    def __init__(self, tokens, vocab, hidden, experts, topk, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.shape = tokens, hidden
        self.ids = torch.randint(-1, vocab, (tokens,), generator=g).cuda()
        self.mask = (self.ids >= 0)
        self.scale = hidden ** 0.5

        def normal(*s, std=1.0):
            return (torch.randn(*s, generator=g) * std).cuda()
        self.p = {"table": normal(vocab, hidden, std=hidden ** -0.5), "router": normal(hidden, experts, std=hidden ** -0.5),
                  "w1": 1 + normal(hidden, std=0.1), "b1": normal(hidden, std=0.1),
                  "w2": 1 + normal(hidden, std=0.1), "b2": normal(hidden, std=0.1),
                  "experts": 1 + normal(experts, 1, std=0.3)}
        self.dy, self.dres = normal(tokens, hidden), normal(tokens, hidden)
        self.rng = torch.tensor([SEED, 0], device="cuda")
        self.dloss = torch.full((1,), 0.7, device="cuda")
        self.plan = ct.MoePlan(tokens, topk, experts)
        t, e, k, rows = tokens, experts, topk, self.plan.rows

        def empty(*s, dtype=F32):
            return torch.empty(*s, dtype=dtype, device="cuda")
        self.b = {n: empty(t, hidden) for n in ("x", "x0", "h", "branch", "res2", "y", "dres2", "dbranch", "dh", "dx", "dx0")}
        self.b.update(xs=empty(rows, hidden), ys=empty(rows, hidden), dys=empty(rows, hidden), dxs=empty(rows, hidden),
                      idx=empty(t, k, dtype=I32), counts=empty(e + 1, dtype=I32), weights=empty(t, k), dweights=empty(t, k),
                      loss=empty(1), logits=empty(t, e), dlogits=empty(t, e), m1=empty(t), r1=empty(t), m2=empty(t), r2=empty(t))
        self.g = {n: torch.empty_like(v) for n, v in self.p.items()}
        u8 = torch.uint8
        self.ws = {"norm": empty(ct.layer_norm_backward_workspace_size(t, hidden), dtype=u8),
                   "router": empty(ct.moe_router_workspace_size(t, k, e), dtype=u8),
                   "table": empty(ct.embedding_backward_workspace_size(t, vocab, hidden), dtype=u8)}

    def expert_of_row(self):
        e = torch.zeros(self.plan.rows, dtype=torch.long, device="cuda")
        slot = self.plan.src.long()
        return torch.where(slot >= 0, self.b["idx"].view(-1)[slot.clamp(min=0)].long(), e)

    def run(self):
        b, p, g = self.b, self.p, self.g
        drop = {"p": P, "rng": self.rng}
        ct.embedding(self.ids, p["table"], b["x"], scale=self.scale)
        ct.dropout(b["x"], b["x0"], P, self.rng, 0)
        ct.layer_norm(None, b["x0"], None, b["h"], p["w1"], p["b1"], EPS, mean=b["m1"], rstd=b["r1"])
        torch.mm(b["h"], p["router"], out=b["logits"])
        ct.moe_router(b["logits"], b["idx"], b["weights"], b["counts"], b["loss"], self.mask, balance=BALANCE, z=Z,
                      workspace=self.ws["router"])
        ct.moe_sort(b["idx"], self.plan)
        ct.moe_dispatch(b["h"], self.plan, b["xs"])
        factor = p["experts"][self.expert_of_row()]
        torch.mul(b["xs"], factor, out=b["ys"])
        ct.moe_combine(b["ys"], self.plan, b["weights"], b["branch"])
        ct.layer_norm(b["branch"], b["x0"], b["res2"], b["y"], p["w2"], p["b2"], EPS, site=1, mean=b["m2"],
                      rstd=b["r2"], **drop)
        # back
        ct.layer_norm_backward(self.dy, self.dres, b["res2"], b["m2"], b["r2"], b["dres2"], b["dbranch"], g["w2"],
                               g["b2"], self.ws["norm"], p["w2"], site=1, **drop)
        ct.moe_combine_backward(b["dbranch"], b["ys"], self.plan, b["weights"], b["dys"], b["dweights"])
        # as a product: torch's index_add_ sums in no fixed order
        of = (self.expert_of_row() == torch.arange(len(p["experts"]), device="cuda")[:, None]).float()
        torch.mm(of, (b["dys"] * b["xs"]).sum(1, keepdim=True), out=g["experts"])
        torch.mul(b["dys"], factor, out=b["dxs"])
        ct.moe_dispatch_backward(b["dxs"], self.plan, b["dh"])
        ct.moe_router_backward(b["dweights"], self.dloss, b["logits"], b["idx"], b["counts"], b["dlogits"], self.mask,
                               balance=BALANCE, z=Z)
        torch.mm(b["h"].t(), b["dlogits"], out=g["router"])
        b["dh"].addmm_(b["dlogits"], p["router"].t())
        ct.layer_norm_backward(b["dh"], b["dres2"], b["x0"], b["m1"], b["r1"], b["dx0"], None, g["w1"], g["b1"],
                               self.ws["norm"], p["w1"])
        ct.dropout(b["dx0"], b["dx"], P, self.rng, 0)
        ct.embedding_backward(self.ids, b["dx"], g["table"], self.ws["table"], scale=self.scale)

    def plain(self, step):
        p = {k: v.detach().double().cpu().requires_grad_() for k, v in self.p.items()}
        ids, mask, idx = self.ids.cpu(), self.mask.cpu(), self.b["idx"].long().cpu()
        f0, f1 = (ref.drop_factor(*self.shape, P, SEED, step, site) for site in (0, 1))

        def norm(x, w, b):
            return (x - x.mean(1, keepdim=True)) * (x.var(1, correction=0, keepdim=True) + EPS).rsqrt() * w + b
        x0 = torch.where(mask[:, None], p["table"][ids.clamp(min=0)] * self.scale, 0.0) * f0
        h = norm(x0, p["w1"], p["b1"])
        logits = h @ p["router"]
        prob, n, k = torch.softmax(logits, 1), int(mask.sum()), idx.shape[1]
        chosen = idx.clamp(min=0)
        weights = torch.softmax(logits.gather(1, chosen), 1) * mask[:, None]
        counts = torch.bincount(idx[mask].view(-1), minlength=prob.shape[1]).double()
        loss = (BALANCE * prob.shape[1] * (counts / (n * k) * prob[mask].mean(0)).sum()
                + Z * torch.logsumexp(logits[mask], 1).square().mean())
        branch = (h[:, None] * p["experts"][chosen][:, :, :] * weights[:, :, None]).sum(1)
        res2 = x0 + branch * f1
        y = norm(res2, p["w2"], p["b2"])
        ((y * self.dy.double().cpu()).sum() + (res2 * self.dres.double().cpu()).sum() + 0.7 * loss).backward()
        return {"y": y, "res2": res2, "loss": loss.view(1)}, {k: v.grad for k, v in p.items()}


def off(got, want):
    got, want = got.detach().double().cpu(), want.detach()
    return ((got - want).norm() / want.norm()).item()


SIZES = [(700, 300, 256, 8, 2), (301, 90, 777, 5, 3), (2000, 5000, 128, 64, 4)]


@pytest.mark.parametrize("sizes", SIZES)
def test_a_step_against_autograd(sizes):
    s = Step(*sizes)
    s.run()
    out, grads = s.plain(0)
    for k, v in out.items():
        assert off(s.b[k], v) < MOST, (k, off(s.b[k], v))
    for k, v in grads.items():
        assert off(s.g[k], v) < MOST, (k, off(s.g[k], v))


@pytest.mark.parametrize("sizes", SIZES[:2])
def test_a_captured_step_is_the_step(sizes):
    """Replays of a graph that moves the generator's step on: each equal to a run of
    its own, bit for bit."""
    s, other = Step(*sizes), Step(*sizes)
    s.run()                                   # what a first call sets up
    s.rng[1] = 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
        s.rng[1:].add_(1)
    s.rng[1] = 0
    for step in range(3):
        graph.replay()
        other.rng[1] = step
        other.run()
        for a, b in ((s.b, other.b), (s.g, other.g)):
            for k in a:
                if k not in ("ys", "dxs", "dys", "xs"):       # padding rows' products
                    assert torch.equal(a[k], b[k]), (step, k)


def test_two_graphs_of_one_stream_each():
    """Two captured steps, replayed at the same time on two streams."""
    steps = [Step(*SIZES[0], seed=i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in steps]
    graphs = []
    for s, stream in zip(steps, streams):
        s.run()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=stream):
            s.run()
    want = [{k: v.clone() for k, v in s.g.items()} for s in steps]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        for k in w:
            assert torch.equal(s.g[k], w[k]), k


def test_a_given_stream():
    """Calls on a stream that is not the current one, behind its own work."""
    rows, hidden = 3000, 2048
    stream = torch.cuda.Stream()
    rng = torch.tensor([1, 2], device="cuda")
    x, out = torch.randn(rows, hidden, device="cuda"), torch.empty(rows, hidden, device="cuda")
    y, z = torch.empty_like(x), torch.empty_like(x)
    ct.dropout(x * 2, y, 0.3, rng, 1)
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(2000000)
        z.copy_(x).mul_(2)
    ct.dropout(z, out, 0.3, rng, 1, stream=stream)
    stream.synchronize()
    assert torch.equal(out, y)
